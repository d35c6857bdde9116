// Attention over the paged 8-bit cache (spark_decode_attn_kv8).
//
// Split-K flash decoding.  The tokens of all (row, kv head) pairs, 32 to a
// step, form one line of steps; each team of warps takes an equal stretch of
// it, whatever the rows' lengths, and walks it with a ring of shared-memory
// stages that TMA fills (keys and values of one step, 8 KB).  A stretch that
// covers a pair wholly writes its output; the others leave (m, l, acc)
// partials that a second kernel merges in order.
//
// Per step and warp, tensor cores (m16n8k16, fp16 in, fp32 out):
//   S^T[token][row]    = K[token][channel] . q^T       codes are exact in fp16
//   O^T[channel][row] += V^T[channel][token] . P^T
// The page's key scale multiplies the scores, its value scale the
// probabilities, so codes are only converted, never scaled.  A query row is
// brought to [2^13, 2^14) by a power of two: bf16 is then exact in fp16
// (elements 2^-27 below the row's largest lose bits), fp32 goes in as two
// fp16 halves.  P is multiplied by 2^14 and by the page's value scale over a
// power of two at or above every scale seen so far, and enters as two fp16
// halves (22 bits, down to 2^-38 of the largest weight), so the result is
// that of fp32 arithmetic.  The codes of values are paired by token with byte
// permutes in registers (the transpose that the second product needs), P is
// transposed by movmatrix; nothing else crosses lanes but the row maxima.
//
// Bound by memory: 256 bytes per token and kv head against about 4.5
// warp-instructions a byte-lane budget of 700 issue slots per 16 tokens.
#include <cuda.h>  // CUtensorMap and its enums (the encoder is fetched at run time)

#include "kv8.cuh"

namespace spark {

bool make_kv8_map(CUtensorMap *tm, const void *codes, long rows, int box_rows);

// Consumer warps of a CTA, for a kernel whose warps work on kNT groups of 8
// query rows; a fourth or third warpgroup holds the producer (one warp works).
// Registers per thread are dealt out from what the launch has (128 or 168):
// 384 * 152 + 128 * 56 = 512 * 128, and 256 * 224 + 128 * 56 = 384 * 168.
constexpr int kMaxTeams = 12;
template <int kNT> struct AtGeom {
    static constexpr int kWarps = kNT == 2 ? 8 : 12;
    static constexpr int kThreads = (kWarps + 4) * 32;
    static constexpr int kRegsConsumer = kNT == 2 ? 224 : 152;
    static constexpr int kRegsProducer = 56;
};
constexpr int kStep = 32;                  // tokens per step
constexpr int kStageBytes = 2 * kStep * kD;
constexpr int kMaxStages = 24;             // stages of a CTA: 192 KB
constexpr int kRingBytes = kMaxStages * kStageBytes;
constexpr int kMinSteps = 2;               // a team takes at least this many steps
constexpr int kPScale = 6;                 // probabilities enter the second product times 2^6
constexpr float kSlack = 8.f;              // log2 of how far a probability may pass its reference

// What a stage's consumers need to know beside the codes.
struct __align__(16) StageMeta {
    float ks[2], vs[2];      // scales of the two halves (16 tokens each)
    int nv[2];               // seen tokens of each half (0 .. 16)
    int b, h;
    int s, n_steps, len;     // step of the row, steps and tokens of the row
    int pad;
};

// workspace: header, the line's layout (int64: steps per team, then steps
// before each row), then partials: acc [slot][rows][128], ml [slot][rows][2]
static size_t attn_layout_bytes(int B) { return (((size_t)B + 1) * 8 + 255) / 256 * 256; }
static long attn_slots(int B, int Hkv, int num_sms) { return (long)num_sms * kMaxTeams + (long)B * Hkv; }

size_t attn_kv8_workspace(int B, int Hkv, int rows, int num_sms) {
    return kWsHeader + attn_layout_bytes(B) + (size_t)attn_slots(B, Hkv, num_sms) * rows * (kD + 2) * sizeof(float);
}

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap *tm, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(row), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ void mma16816(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Four codes -> two fp16 pairs: codes (0, 1) and (2, 3).
template <int kType> __device__ __forceinline__ void expand4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if (kType == SPARK_KV8_E4M3) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        // 0x6400 | (code + 128) is the fp16 number 1024 + 128 + code
        const uint32_t u = w ^ 0x80808080u;
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
        uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off);
        const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
        lo = *reinterpret_cast<const uint32_t *>(&x);
        hi = *reinterpret_cast<const uint32_t *>(&y);
    }
}

// 0xff in each byte that is an e4m3 NaN (0x7f or 0xff).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
    return ((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu;
}

// A place on the line of steps.
struct Place {
    int b, h, s;       // row, kv head, step of the row
    int len, n_steps;  // tokens and steps of the row
};

struct AttnArgs {
    spark_kv8cache kc;
    const int32_t *table, *lens, *n_new;
    int table_cap, B, rows, n_q, team_warps, n_stages;
    float *out;
    uint32_t *ws;
    long long *layout;
    float *acc, *ml;
};

__device__ __forceinline__ int clamped_len(const AttnArgs &a, int b) {
    return min(max(__ldg(a.lens + b), 0), a.table_cap * a.kc.page);
}

__device__ __forceinline__ void set_row(const AttnArgs &a, Place &p, int b) {
    p.b = b;
    p.len = clamped_len(a, b);
    p.n_steps = (p.len + kStep - 1) / kStep;
}

// The pair after p's (rows without tokens have no steps).
__device__ __forceinline__ void next_pair(const AttnArgs &a, Place &p) {
    p.s = 0;
    if (++p.h < a.kc.Hkv) return;
    p.h = 0;
    do set_row(a, p, p.b + 1);
    while (p.n_steps == 0);
}

// One step as the producer sees it: the pages of its halves, then their scales.
struct StepLoad {
    Place p;
    int pg[2];
    float ks[2], vs[2];
};

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) { return mbar_try_wait(bar, parity); }

// kNT: 8-row groups a warp works on; 0: up to 4 rows, whose second copy in
// the group's other 4 places carries P's low halves through the same product.
template <typename E, int kType, int kNT>
__global__ void __launch_bounds__(AtGeom<kNT>::kThreads, 1)
    attn_kv8_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    const E *__restrict__ q, const AttnArgs a) {
    constexpr int kAtWarps = AtGeom<kNT>::kWarps, kAtThreads = AtGeom<kNT>::kThreads;
    constexpr int kN = kNT ? kNT : 1;              // 8-row groups
    constexpr int kRows = kNT ? 8 * kNT : 4;       // query rows of a warp
    constexpr int kQ = sizeof(E) == 4 ? 2 : 1;     // fp16 halves of a query
    extern __shared__ unsigned char sm_raw[];
    __shared__ long long before[kAtThreads + 1];   // steps (of one kv head) before each thread's rows
    __shared__ long long wsum[kAtThreads / 32];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages];
    __shared__ StageMeta meta[kMaxStages];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int tw = a.team_warps, n_teams = kAtWarps / tw, team = warp / tw, wt = warp % tw;
    const int Hkv = a.kc.Hkv, ns = a.n_stages;
    const uint32_t ring = (smem_u32(sm_raw) + 1023u) & ~1023u;

    // ---- the line: steps before each thread's rows, and in all
    const int per = (a.B + kAtThreads - 1) / kAtThreads;
    {
        long long mine = 0;
        bool bad = false;
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            if (b < a.B) {
                const int len = clamped_len(a, b), nn = a.n_new ? __ldg(a.n_new + b) : a.n_q;
                bad |= len != __ldg(a.lens + b) || nn < 0 || nn > a.n_q;
                mine += (len + kStep - 1) / kStep;
            }
        }
        if (bad && blockIdx.x == 0) atomicOr(a.ws, kDevBadArg);
        long long v = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += y;
        }
        if (lane == 31) wsum[warp] = v;
        if (tid < kMaxStages) {
            mbar_init(smem_u32(&full[tid]), 1);
            mbar_init(smem_u32(&empty[tid]), tw);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncthreads();
        long long pre = 0;
        for (int w = 0; w < warp; ++w) pre += wsum[w];
        before[tid + 1] = pre + v;
        if (tid == 0) before[0] = 0;
        __syncthreads();
        if (blockIdx.x == 0) {  // for the merge
            long long x = before[tid];
            for (int i = 0; i < per; ++i) {
                const int b = tid * per + i;
                if (b < a.B) {
                    a.layout[1 + b] = x;
                    x += (clamped_len(a, b) + kStep - 1) / kStep;
                }
            }
        }
    }
    const long long total = before[kAtThreads] * Hkv;
    const long long all_teams = (long long)gridDim.x * n_teams;
    const long long share = max((total + all_teams - 1) / all_teams, (long long)kMinSteps);
    if (blockIdx.x == 0 && tid == 0) a.layout[0] = share;

    if (warp >= kAtWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(AtGeom<kNT>::kRegsProducer));
        if (warp > kAtWarps) return;
        // ---- producer: lane t keeps team t's part of the ring full
        const long long from = ((long long)blockIdx.x * n_teams + lane) * share;
        int left = lane < n_teams && from < total ? (int)min(share, total - from) : 0;
        bool bad = false;
        const int page = a.kc.page, shift = 31 - __clz(page);
        StepLoad d0, d1;
        Place pl = {0, 0, 0, 0, 0};
        int to_load = left;
        // pages of the next step that has none yet
        auto load_pages = [&](StepLoad &d) {
            d.pg[0] = d.pg[1] = -1;
            if (to_load == 0) return;
            if (pl.s == pl.n_steps) next_pair(a, pl);
            d.p = pl;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tok = pl.s * kStep + i * 16;
                if (tok < pl.len) d.pg[i] = __ldg(a.table + (size_t)pl.b * a.table_cap + (tok >> shift));
            }
            ++pl.s;
            --to_load;
        };
        auto load_scales = [&](StepLoad &d) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                d.ks[i] = d.vs[i] = 0.f;
                const bool ok = (unsigned)d.pg[i] < (unsigned)a.kc.n_pages;
                if (ok) {
                    d.ks[i] = __ldg(a.kc.k_scale + (size_t)d.pg[i] * Hkv + d.p.h);
                    d.vs[i] = __ldg(a.kc.v_scale + (size_t)d.pg[i] * Hkv + d.p.h);
                }
            }
        };
        if (left > 0) {
            int lo = 0, hi = kAtThreads;  // the last thread whose rows start at or before `from`
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (before[mid] * Hkv <= from) lo = mid;
                else hi = mid;
            }
            long long pos = from - before[lo] * Hkv;
            for (int b = lo * per;; ++b) {
                set_row(a, pl, b);
                if (pos < (long long)pl.n_steps * Hkv) break;
                pos -= (long long)pl.n_steps * Hkv;
            }
            pl.h = (int)(pos / pl.n_steps);
            pl.s = (int)(pos % pl.n_steps);
            load_pages(d0);
            load_scales(d0);
            load_pages(d1);
        }
        const int st0 = lane * ns;
        int st = 0;
        uint32_t parity = 1;  // a fresh barrier passes
        uint64_t since = global_ns();
        bool failed = false;
        while (__any_sync(0xffffffffu, left > 0)) {
            const bool ready = left > 0 && mbar_test(smem_u32(&empty[st0 + st]), parity);
            if (ready) {
                const int tok = d0.p.s * kStep, len = d0.p.len;
                bool ok[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ok[i] = (unsigned)d0.pg[i] < (unsigned)a.kc.n_pages;
                    bad |= !ok[i] && tok + i * 16 < len;
                }
                StageMeta &m = meta[st0 + st];
                m.ks[0] = d0.ks[0];
                m.ks[1] = d0.ks[1];
                m.vs[0] = d0.vs[0];
                m.vs[1] = d0.vs[1];
                m.nv[0] = ok[0] ? min(16, len - tok) : 0;
                m.nv[1] = ok[1] ? min(16, len - tok - 16) : 0;
                m.b = d0.p.b;
                m.h = d0.p.h;
                m.s = d0.p.s;
                m.n_steps = d0.p.n_steps;
                m.len = len;
                const uint32_t bar = smem_u32(&full[st0 + st]), dst = ring + (uint32_t)(st0 + st) * kStageBytes;
                if (page >= kStep) {
                    mbar_expect_tx(bar, ok[0] ? 2 * kStep * kD : 0);
                    if (ok[0]) {
                        const int row = (d0.pg[0] * Hkv + d0.p.h) * page + (tok & (page - 1));
                        tma_rows(dst, &map_k, row, bar);
                        tma_rows(dst + kStep * kD, &map_v, row, bar);
                    }
                } else {
                    mbar_expect_tx(bar, (ok[0] + ok[1]) * 2 * 16 * kD);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (ok[i]) {
                            const int row = (d0.pg[i] * Hkv + d0.p.h) * 16;
                            tma_rows(dst + i * 16 * kD, &map_k, row, bar);
                            tma_rows(dst + (kStep + i * 16) * kD, &map_v, row, bar);
                        }
                }
                --left;
                if (++st == ns) {
                    st = 0;
                    parity ^= 1;
                }
                d0 = d1;
                load_scales(d0);
                load_pages(d1);
            }
            if (__any_sync(0xffffffffu, ready)) {
                since = global_ns();
            } else {
                __nanosleep(40);
                if (global_ns() - since > 1000000000ull) {
                    failed = true;
                    break;
                }
            }
        }
        if (bad) atomicOr(a.ws, kDevBadArg);
        if (failed) {
            // some consumer gave up; let the copies in flight land before the CTA's memory goes away
            if (lane == 0) atomicOr(a.ws, kDevTimeout);
            if (lane < n_teams)
                for (int i = 0; i < ns; ++i) {
                    const int u = (st + i) % ns;  // its last use had this parity (of a stage never used, 1: passes)
                    mbar_wait_bounded(smem_u32(&full[st0 + u]), st + i < ns ? parity : parity ^ 1u);
                }
        }
        return;
    }

    // ---- consumers
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(AtGeom<kNT>::kRegsConsumer));
    if (team >= n_teams) return;  // warps that make no whole team
    const long long tm = (long long)blockIdx.x * n_teams + team;
    const long long from = tm * share;
    if (from >= total) return;
    const int steps = (int)min(share, total - from);
    const int st0 = team * ns;
    const uint32_t base = ring + (uint32_t)st0 * kStageBytes;

    uint32_t qh[kQ][kN][16];      // B fragments of the queries
    float qf[kN][2];              // score factor of rows 2c, 2c + 1
    int lim[kN][2];               // the last token they see
    float o[kN][8][4], m[kN][2], l[kN][2];
    float E_top = 1.f, E_inv = 1.f;
    int b = -1, h = 0, nn = 0, first_full = 0;
    bool starts_pair = false, ends_pair = false;
    auto begin_pair = [&](const StageMeta &mt) {
        b = mt.b;
        h = mt.h;
        nn = a.n_new ? min(max(__ldg(a.n_new + b), 0), a.n_q) : a.n_q;
        first_full = mt.len - nn + 1;  // tokens below this are seen by every query
        starts_pair = mt.s == 0;
        E_top = exp2_int(-100);
        E_inv = exp2_int(100 + kPScale);
        const E *qb = q + ((size_t)b * Hkv + h) * a.rows * kD;
#pragma unroll
        for (int t = 0; t < kN; ++t) {
            const int r = wt * kRows + (kNT ? t * 8 + g : (g & 3));
            float x[32], top = 0.f;
            if (r < a.rows) {
                const uint4 *src = reinterpret_cast<const uint4 *>(qb + (size_t)r * kD + c * 32);
#pragma unroll
                for (int i = 0; i < (int)sizeof(E) * 2; ++i) {
                    const uint4 u = __ldg(src + i);
                    const E *e = reinterpret_cast<const E *>(&u);
#pragma unroll
                    for (int j = 0; j < 16 / (int)sizeof(E); ++j) x[i * (16 / (int)sizeof(E)) + j] = Elem<E>::to_f(e[j]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(x[i]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int fe = min(13 - ((int)(__float_as_uint(top) >> 23) - 127), 126);  // -115 .. 126
            const float f = exp2_int(fe);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float y0 = x[2 * i] * f, y1 = x[2 * i + 1] * f;
                const __half2 hi = __floats2half2_rn(y0, y1);
                qh[0][t][i] = *reinterpret_cast<const uint32_t *>(&hi);
                if (kQ == 2) {
                    const float2 back = __half22float2(hi);
                    qh[kQ - 1][t][i] = pack_half2(y0 - back.x, y1 - back.y);
                }
            }
            const float mine = exp2_int(-fe) * (float)(1.4426950408889634 / 11.313708498984761);  // log2 e / sqrt(D)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                qf[t][j] = __shfl_sync(0xffffffffu, mine, (2 * c + j) * 4);
                const int col = kNT ? t * 8 + 2 * c + j : (2 * c + j) & 3;
                const int row = wt * kRows + col, i = row % a.n_q;
                lim[t][j] = row < a.rows && i < nn ? mt.len - nn + i : -1;
                m[t][j] = -INFINITY;
                l[t][j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.f;
        }
    };
    auto end_pair = [&]() {
        const long bh = (long)b * Hkv + h;
        const bool whole = starts_pair && ends_pair;
#pragma unroll
        for (int t = 0; t < kN; ++t) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float s = l[t][j];
                s += __shfl_xor_sync(0xffffffffu, s, 4);
                s += __shfl_xor_sync(0xffffffffu, s, 8);
                s += __shfl_xor_sync(0xffffffffu, s, 16);
                l[t][j] = s;
            }
            if (kNT == 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[t][j][i] += __shfl_xor_sync(0xffffffffu, o[t][j][i], 2);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = kNT ? t * 8 + 2 * c + j : (2 * c + j) & 3;
                const int row = wt * kRows + col;
                if ((kNT == 0 && c >= 2) || row >= a.rows || row % a.n_q >= nn) continue;
                float *dst;
                float f = E_top * exp2_int(-kPScale);
                if (whole) {
                    dst = a.out + (bh * a.rows + row) * kD;
                    f = l[t][j] == 0.f ? 0.f : f / l[t][j];
                } else {
                    const size_t at = (size_t)(tm + bh) * a.rows + row;
                    dst = a.acc + at * kD;
                    if (g == 0) *reinterpret_cast<float2 *>(a.ml + at * 2) = make_float2(m[t][j], l[t][j]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float4 *>(dst + g * 16 + i * 4) =
                        make_float4(o[t][2 * i][j] * f, o[t][2 * i][2 + j] * f, o[t][2 * i + 1][j] * f,
                                    o[t][2 * i + 1][2 + j] * f);
            }
        }
    };

    int st = 0;
    uint32_t parity = 0;
    for (int it = 0; it < steps; ++it) {
        if (!mbar_wait_bounded(smem_u32(&full[st0 + st]), parity)) {
            if (lane == 0) atomicOr(a.ws, kDevTimeout);
            return;
        }
        const StageMeta mt = meta[st0 + st];
        if (mt.b != b || mt.h != h) {
            if (b >= 0) end_pair();
            begin_pair(mt);
        }
        ends_pair = mt.s + 1 == mt.n_steps;
        const uint32_t kb = base + (uint32_t)st * kStageBytes, vb = kb + kStep * kD;
        const int t0 = mt.s * kStep;

        // scores
        float s[kN][2][4];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int t = 0; t < kN; ++t) s[t][hf][0] = s[t][hf][1] = s[t][hf][2] = s[t][hf][3] = 0.f;
            const uint32_t r0 = kb + (uint32_t)(hf * 16 + g) * kD;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t x = (uint32_t)((2 * c + i) ^ g) << 4;
                const uint4 u = lds128(r0 + x), w = lds128(r0 + 8 * kD + x);
                const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t a0, a1, a2, a3;
                    expand4<kType>(uu[j], a0, a2);
                    expand4<kType>(ww[j], a1, a3);
                    const int f = (i * 4 + j) * 2;
#pragma unroll
                    for (int t = 0; t < kN; ++t)
#pragma unroll
                        for (int y = 0; y < kQ; ++y)
                            mma16816(s[t][hf], a0, a1, a2, a3, qh[y][t][f], qh[y][t][f + 1]);
                }
            }
        }
        // places without a token and tokens behind a query's own
        const bool edge = mt.nv[0] < 16 || mt.nv[1] < 16 || t0 + kStep > first_full;
        bool hide = false;
        if (edge) {
#pragma unroll
            for (int t = 0; t < kN; ++t)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int in = g + 8 * (i >> 1);
                        if (in >= mt.nv[hf] || t0 + hf * 16 + in > lim[t][i & 1]) s[t][hf][i] = -INFINITY;
                    }
            // Places without a token may hold anything, NaN codes too: their
            // values become zeros before the second product meets them.
            if (mt.nv[0] < 16 || mt.nv[1] < 16) {
                for (int i = lane; i < kStep * 8; i += 32) {
                    const int row = i >> 3;
                    if ((row & 15) >= (row < 16 ? mt.nv[0] : mt.nv[1]))
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vb + (uint32_t)i * 16), "r"(0u)
                                     : "memory");
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            // A token that some of the queries do not see takes part in the second
            // product with p = 0 for them: where its value is NaN, the queries that
            // see it get their NaN here and the product a zero.
            if (kType == SPARK_KV8_E4M3 && a.n_q > 1) {
#pragma unroll 1
                for (int i = max(first_full - t0, 0); i < kStep; ++i) {
                    if ((i & 15) >= (i < 16 ? mt.nv[0] : mt.nv[1])) continue;
                    const uint4 w = lds128(vb + (uint32_t)i * kD + ((uint32_t)(g ^ (i & 7)) << 4));
                    const uint32_t ww[4] = {nan_codes(w.x), nan_codes(w.y), nan_codes(w.z), nan_codes(w.w)};
                    if (!__any_sync(0xffffffffu, (ww[0] | ww[1] | ww[2] | ww[3]) != 0)) continue;
                    hide = true;
#pragma unroll
                    for (int t = 0; t < kN; ++t)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
#pragma unroll
                            for (int y = 0; y < 2; ++y)
                                if (((ww[j / 4] >> (8 * (j % 4))) & 0xffu) && t0 + i <= lim[t][y])
                                    o[t][j / 2][(j & 1) * 2 + y] = __int_as_float(0x7fffffff);
                }
            }
        }
        // The reference m of a row's probabilities (in units of log2) is its
        // largest score so far, but follows it only when that is more than
        // kSlack above: the sums take any reference, and most steps then
        // need no maximum across lanes and no rescaling.
        float f[kN][2][2];
        bool move = false;
#pragma unroll
        for (int t = 0; t < kN; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // above 0, so that an unseen place stays at -inf whatever its page's scale
                f[t][0][j] = fmaxf(qf[t][j] * mt.ks[0], exp2_int(-126));
                f[t][1][j] = fmaxf(qf[t][j] * mt.ks[1], exp2_int(-126));
                const float mx = fmaxf(fmaxf(s[t][0][j], s[t][0][2 + j]) * f[t][0][j],
                                       fmaxf(s[t][1][j], s[t][1][2 + j]) * f[t][1][j]);
                move |= mx > m[t][j] + kSlack;
            }
        const float vm = fmaxf(mt.vs[0], mt.vs[1]);
        if (__any_sync(0xffffffffu, move || vm > E_top)) {
            float grow = 1.f;
            if (vm > E_top) {
                const float top = __uint_as_float((__float_as_uint(vm) & 0x7f800000u) + 0x800000u);
                grow = E_top / top;
                E_top = top;
                E_inv = exp2_int(kPScale) / top;
            }
#pragma unroll
            for (int t = 0; t < kN; ++t) {
                float al[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float mx = fmaxf(fmaxf(s[t][0][j], s[t][0][2 + j]) * f[t][0][j],
                                     fmaxf(s[t][1][j], s[t][1][2 + j]) * f[t][1][j]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float mn = fmaxf(m[t][j], mx);
                    al[j] = mn > m[t][j] ? exp2_approx(m[t][j] - mn) : 1.f;  // 0 from -inf
                    m[t][j] = mn;
                    l[t][j] *= al[j];
                    al[j] *= grow;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    o[t][j][0] *= al[0];
                    o[t][j][1] *= al[1];
                    o[t][j][2] *= al[0];
                    o[t][j][3] *= al[1];
                }
            }
        }
        // probabilities, their sums, and the second product
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const float cf = mt.vs[hf] * E_inv;
            uint32_t ph[kN][2], pl_[kN][2];
#pragma unroll
            for (int t = 0; t < kN; ++t) {
                const float m0 = m[t][0] == -INFINITY ? 0.f : m[t][0], m1 = m[t][1] == -INFINITY ? 0.f : m[t][1];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float p0 = exp2_approx(s[t][hf][2 * r] * f[t][hf][0] - m0);
                    float p1 = exp2_approx(s[t][hf][2 * r + 1] * f[t][hf][1] - m1);
                    l[t][0] += p0;
                    l[t][1] += p1;
                    p0 *= cf;
                    p1 *= cf;
                    const __half2 hi = __floats2half2_rn(p0, p1);
                    const float2 back = __half22float2(hi);
                    const uint32_t hb = *reinterpret_cast<const uint32_t *>(&hi);
                    const uint32_t lb = pack_half2(p0 - back.x, p1 - back.y);
                    if (kNT == 0) {
                        ph[t][r] = transpose8x8(c < 2 ? hb : lb);
                    } else {
                        ph[t][r] = transpose8x8(hb);
                        pl_[t][r] = transpose8x8(lb);
                    }
                }
            }
            // lane (g, c): tokens 2c, 2c + 1, 2c + 8, 2c + 9, channels 16 g .. 16 g + 15
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = hf * 16 + 2 * c + (i & 1) + (i >> 1) * 8;
                w[i] = lds128(vb + (uint32_t)row * kD + ((uint32_t)(g ^ (row & 7)) << 4));
                if (kType == SPARK_KV8_E4M3 && hide && t0 + row >= first_full)
                    w[i] = make_uint4(w[i].x & ~nan_codes(w[i].x), w[i].y & ~nan_codes(w[i].y),
                                      w[i].z & ~nan_codes(w[i].z), w[i].w & ~nan_codes(w[i].w));
            }
            const uint32_t ww[4][4] = {{w[0].x, w[0].y, w[0].z, w[0].w}, {w[1].x, w[1].y, w[1].z, w[1].w},
                                       {w[2].x, w[2].y, w[2].z, w[2].w}, {w[3].x, w[3].y, w[3].z, w[3].w}};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t a0, a1, a2, a3;
                    expand4<kType>(__byte_perm(ww[0][j], ww[1][j], y ? 0x7362 : 0x5140), a0, a1);
                    expand4<kType>(__byte_perm(ww[2][j], ww[3][j], y ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                    for (int t = 0; t < kN; ++t) {
                        mma16816(o[t][2 * j + y], a0, a1, a2, a3, ph[t][0], ph[t][1]);
                        if (kNT) mma16816(o[t][2 * j + y], a0, a1, a2, a3, pl_[t][0], pl_[t][1]);
                    }
                }
            }
        }
        // the stage is free once every warp of the team has read it
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&empty[st0 + st]));
        if (++st == ns) {
            st = 0;
            parity ^= 1;
        }
    }
    end_pair();
}

// Merge of the partials of one query row: CTA = row, warps take partials in
// turn, and their results are added in warp order.
constexpr int kMgWarps = 8;

__global__ void __launch_bounds__(kMgWarps * 32) attn_kv8_merge_kernel(const AttnArgs a) {
    __shared__ float4 acc_s[kMgWarps][32];
    __shared__ float m_s[kMgWarps], l_s[kMgWarps];
    const long bh = blockIdx.x / a.rows;
    const int row = blockIdx.x % a.rows, b = (int)(bh / a.kc.Hkv), h = (int)(bh % a.kc.Hkv);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nn = a.n_new ? min(max(__ldg(a.n_new + b), 0), a.n_q) : a.n_q;
    if (row % a.n_q >= nn) return;
    float *out = a.out + (bh * a.rows + row) * kD;
    const int n_steps = (clamped_len(a, b) + kStep - 1) / kStep;
    if (n_steps == 0) {
        if (warp == 0) *reinterpret_cast<float4 *>(out + lane * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    const long long share = a.layout[0], first = a.layout[1 + b] * a.kc.Hkv + (long long)h * n_steps;
    const long long t0 = first / share, t1 = (first + n_steps - 1) / share;
    if (t0 == t1) return;  // written by the one team that had it all
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (long long t = t0 + warp; t <= t1; t += kMgWarps) {
        const size_t at = (size_t)(t + bh) * a.rows + row;
        const float2 x = *reinterpret_cast<const float2 *>(a.ml + at * 2);
        const float4 v = *reinterpret_cast<const float4 *>(a.acc + at * kD + lane * 4);
        const float mn = fmaxf(m, x.x);
        const float f = mn == -INFINITY ? 1.f : exp2_approx(m - mn), e = mn == -INFINITY ? 1.f : exp2_approx(x.x - mn);
        l = l * f + x.y * e;
        acc = make_float4(acc.x * f + v.x * e, acc.y * f + v.y * e, acc.z * f + v.z * e, acc.w * f + v.w * e);
        m = mn;
    }
    acc_s[warp][lane] = acc;
    if (lane == 0) {
        m_s[warp] = m;
        l_s[warp] = l;
    }
    __syncthreads();
    if (warp) return;
    m = -INFINITY;
    for (int i = 0; i < kMgWarps; ++i) m = fmaxf(m, m_s[i]);
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < kMgWarps; ++i) {
        const float e = m == -INFINITY ? 1.f : exp2_approx(m_s[i] - m);
        const float4 v = acc_s[i][lane];
        l += l_s[i] * e;
        acc = make_float4(acc.x + v.x * e, acc.y + v.y * e, acc.z + v.z * e, acc.w + v.w * e);
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<float4 *>(out + lane * 4) = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
}

template <typename E, int kType, int kNT>
static cudaError_t launch_one(const CUtensorMap &mk, const CUtensorMap &mv, const void *q, const AttnArgs &a,
                              int num_sms, cudaStream_t st) {
    const size_t smem = kRingBytes + 1024;
    auto kernel = attn_kv8_kernel<E, kType, kNT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)num_sms, AtGeom<kNT>::kThreads, smem, st>>>(mk, mv, static_cast<const E *>(q), a);
    return cudaGetLastError();
}

template <typename E, int kType>
static cudaError_t launch_rows(const CUtensorMap &mk, const CUtensorMap &mv, const void *q, AttnArgs &a, int num_sms,
                               cudaStream_t st) {
    // rows a warp works on; two groups of 8 only for bf16 queries, whose fragments take half the registers
    const int per = a.rows <= 4 ? 4 : (a.rows <= 8 || sizeof(E) == 4) ? 8 : 16;
    a.team_warps = (a.rows + per - 1) / per;
    const int teams = (per == 16 ? AtGeom<2>::kWarps : AtGeom<1>::kWarps) / a.team_warps;
    a.n_stages = min(kMaxStages / teams, 8);
    if (per == 4) return launch_one<E, kType, 0>(mk, mv, q, a, num_sms, st);
    if (per == 8) return launch_one<E, kType, 1>(mk, mv, q, a, num_sms, st);
    return launch_one<E, kType, sizeof(E) == 4 ? 1 : 2>(mk, mv, q, a, num_sms, st);
}

cudaError_t launch_attn_kv8(const void *q, int dtype, const spark_kv8cache &kc, const int32_t *table, int table_cap,
                            const int32_t *lens, const int32_t *n_new, int B, int G, int n_q, float *out, void *ws,
                            int num_sms, cudaStream_t st) {
    AttnArgs a;
    a.kc = kc;
    a.table = table;
    a.lens = lens;
    a.n_new = n_new;
    a.table_cap = table_cap;
    a.B = B;
    a.rows = G * n_q;
    a.n_q = n_q;
    a.out = out;
    char *w = static_cast<char *>(ws);
    a.ws = reinterpret_cast<uint32_t *>(w);
    a.layout = reinterpret_cast<long long *>(w + kWsHeader);
    a.acc = reinterpret_cast<float *>(w + kWsHeader + attn_layout_bytes(B));
    a.ml = a.acc + (size_t)attn_slots(B, kc.Hkv, num_sms) * a.rows * kD;
    CUtensorMap mk, mv;
    const long rows = (long)kc.n_pages * kc.Hkv * kc.page;
    // a pool without pages is never read: any address does
    if (!make_kv8_map(&mk, rows ? kc.k : ws, rows ? rows : 1, kc.page < kStep ? kc.page : kStep) ||
        !make_kv8_map(&mv, rows ? kc.v : ws, rows ? rows : 1, kc.page < kStep ? kc.page : kStep))
        return cudaErrorInvalidValue;
    const bool e4 = kc.type == SPARK_KV8_E4M3;
    cudaError_t e;
    if (dtype == SPARK_F32)
        e = e4 ? launch_rows<float, SPARK_KV8_E4M3>(mk, mv, q, a, num_sms, st)
               : launch_rows<float, SPARK_KV8_I8>(mk, mv, q, a, num_sms, st);
    else
        e = e4 ? launch_rows<__nv_bfloat16, SPARK_KV8_E4M3>(mk, mv, q, a, num_sms, st)
               : launch_rows<__nv_bfloat16, SPARK_KV8_I8>(mk, mv, q, a, num_sms, st);
    if (e != cudaSuccess) return e;
    attn_kv8_merge_kernel<<<(unsigned)((long)B * kc.Hkv * a.rows), kMgWarps * 32, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace spark
