// Attention over the paged 8-bit cache (spark_decode_attn_kv8).
//
// Split-K flash decoding in one launch, one CTA per SM.  The tokens of all
// (row, kv head) pairs, 32 to a step, form one line of steps, row after row;
// each CTA takes an equal stretch of it and each of its teams an equal part of
// that, whatever the rows' lengths (48 rows of 17 to 32768 tokens run at the
// rate of equal ones).  A team is as many warps as the query rows need, and
// keeps a ring of stages that TMA fills (keys and values of a step, 8 KB, in
// the 128-byte swizzle, which makes every fragment load below conflict-free).
//
// Per step and warp, tensor cores (m16n8k16, fp16 in, fp32 out):
//   S^T[token][row]    = K[token][channel] . q^T       codes are exact in fp16
//   O^T[channel][row] += V^T[channel][token] . P^T
// The page's key scale multiplies the scores, its value scale the
// probabilities, so codes are only converted, never scaled.  A query row is
// brought to [2^13, 2^14) by a power of two: bf16 is then exact in fp16
// (elements 2^-27 below the row's largest lose bits), fp32 goes in as two
// fp16 halves (22 bits).  P is multiplied by the page's value scale and 2^6
// over a power of two that follows the row's largest product of the two, and
// enters as two fp16 halves: 22 bits, down to 2^-29 of that product, however
// far the value scales of a row lie apart.  The sums come out with the error of
// fp32 ones.  The codes of values are paired by token with byte permutes
// in registers (the transpose that the second product needs), P is transposed
// by movmatrix; nothing else crosses lanes but the row maxima.
//
// A pair that one team has wholly is written at once.  Of others the teams
// leave (m, l, acc) partials, which their CTA merges from shared memory; where
// a pair crosses CTAs, the last of them to finish merges the CTAs' partials,
// always in their order, so that results do not depend on timing.
//
// tcgen05 was not taken: a decode step has 4 to 16 query rows per kv head,
// and codes would have to go through registers and back to shared memory as
// fp16 first.  Legacy matrix instructions take their operands from registers,
// where the codes are converted anyway, and are 17 % busy at 4 rows.
//
// Bound, from the profile: at up to 8 rows by memory while the ring is full
// (about 23 bytes a clock and SM, 90 % of the copy rate between the first
// stage's arrival and the last step), with 2.6 us before it (lengths, their
// sum, table, pages: four dependent reads) and 4 to 8 us behind it (slowest
// SM, merges).  At 16 rows by dependent-issue latency: some 250 registers leave 8
// warps, issue slots are 35 % used, and 77 us of 4 verified tokens compare
// with 41 us of memory time.
#include <cuda.h>  // CUtensorMap and its enums (the encoder is fetched at run time)

#include "kv8.cuh"

namespace spark {

bool make_kv8_map(CUtensorMap *tm, const void *codes, long rows, int box_rows);

// Warps of a CTA, for a kernel whose warps work on kNT groups of 8 query rows
// (168 or 255 registers a thread).  8 warps instead of 12 at kNT = 0 and 1: 3 to
// 5 % slower; 12 at kNT = 2: spills, 109 us instead of 78.
constexpr int kMaxTeams = 12;
template <int kNT> struct AtGeom {
    static constexpr int kWarps = kNT == 2 ? 8 : 12;
    static constexpr int kThreads = kWarps * 32;
};
constexpr int kStep = 32;                  // tokens per step
constexpr int kStageBytes = 2 * kStep * kD;
constexpr int kMaxStages = 24;             // stages of a CTA: 192 KB
constexpr int kRingBytes = kMaxStages * kStageBytes;
constexpr int kMinCtaSteps = 4;            // a CTA takes at least this many steps
constexpr int kPScale = 6;                 // the row's largest p * value scale enters the second product near 2^6
constexpr float kSlack = 5.f;              // log2 of how far a probability may pass its reference
constexpr float kTopFactor = 1024.f;       // value scale * 2^6 / E up to which p <= 2^kSlack stays in fp16
constexpr int kMinE = -120, kMaxE = 126;   // 2^(6 - E) and 2^(E - 6) are normal fp32

// What a stage's consumers need to know beside the codes.
struct __align__(16) StageMeta {
    float ks[2], vs[2];      // scales of the two halves (16 tokens each)
    int nv[2];               // seen tokens of each half (0 .. 16)
    int b, h;
    int s, n_steps, len;     // step of the row, steps and tokens of the row
    int pad;
};

// Workspace: header, one counter per CTA (zero between calls), the warps'
// flushed sums ([warp][9 * kN][lane] float4), then the partials of teams and
// of CTAs: acc [slot][rows][128] fp32, and (m, l) [slot][rows][2].  Along the
// line the team and the pair only grow, so team + pair numbers a team's
// partial of a pair uniquely, and CTA + pair a CTA's.
static size_t attn_counter_bytes(int num_sms) { return ((size_t)num_sms * 4 + 255) / 256 * 256; }
// of a CTA: 8 warps with two 8-row groups (12 with one need less)
constexpr size_t kFlushBytes = 8 * 2 * 9 * 32 * sizeof(float4);
static long attn_team_slots(long pairs, int num_sms) { return (long)num_sms * kMaxTeams + pairs; }

size_t attn_kv8_workspace(int B, int Hkv, int rows, int num_sms) {
    const long pairs = (long)B * Hkv;
    const size_t slots = (size_t)(attn_team_slots(pairs, num_sms) + num_sms + pairs);
    return kWsHeader + attn_counter_bytes(num_sms) + num_sms * kFlushBytes + slots * rows * (kD + 2) * sizeof(float);
}

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap *tm, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(row), "r"(bar)
        : "memory");
}

// A value that is the same in all lanes, in a form from which the compiler
// knows that.  One branch in a loop whose condition may differ between lanes
// for all the compiler knows (a loaded number, say), with a shuffle or a vote
// behind it, and every shuffle, vote and transpose of the loop becomes a
// call-like sequence of some 200 cycles.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool uniform(bool x) { return __any_sync(0xffffffffu, x) != 0; }

// The same value, of which the compiler knows nothing.  Conditions on launch
// constants inside the main loop go through this: the compiler would make a
// copy of the whole loop for each outcome of each of them, and what a CTA runs
// once costs what its fetch costs.
__device__ __forceinline__ int opaque(int x) {
    asm volatile("" : "+r"(x));
    return x;
}

// Bounded wait of a whole warp (about 1 s); the answer is the same in all
// lanes.  Written without unrolling: it is code that every CTA fetches.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
    bool ok = mbar_try_wait(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        const uint64_t since = global_ns();
#pragma unroll 1
        for (uint32_t it = 0; !ok && it < (1u << 26); ++it) {
            ok = mbar_try_wait(bar, parity);
            if ((it & 63u) == 63u && global_ns() - since > 1000000000ull) break;
        }
    }
    return __all_sync(0xffffffffu, ok);
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

// 1 / x for a power of two; 2^127 for 0 (it then multiplies zeros).
__device__ __forceinline__ float inverse_pow2(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }

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

__device__ __forceinline__ uint32_t add_acq_rel(uint32_t *p) {
    uint32_t r;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(r) : "l"(p) : "memory");
    return r;
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
    uint32_t *ws, *counter;
    float4 *flush;          // flushed sums
    float *acc, *ml;        // team partials
    float *acc_c, *ml_c;    // CTA partials
};

__device__ __forceinline__ int clamped_len(const AttnArgs &a, int b) {
    return min(max(a.lens[b], 0), a.table_cap * a.kc.page);
}

// 32-bit sums that pass a row's or the line's end (both below 2^31) are unsigned.
__device__ __forceinline__ int steps_of(int len) { return (int)(((unsigned)len + (kStep - 1)) / kStep); }

__device__ __forceinline__ void set_row(const AttnArgs &a, Place &p, int b) {
    p.b = b;
    p.len = clamped_len(a, b);
    p.n_steps = steps_of(p.len);
}

// The pair after p's (rows without tokens have no steps).
__device__ __forceinline__ void next_pair(const AttnArgs &a, Place &p) {
    p.s = 0;
    if (++p.h < a.kc.Hkv) return;
    p.h = 0;
#pragma unroll 1
    do {
        set_row(a, p, p.b + 1);
        p.len = uniform(p.len);
        p.n_steps = uniform(p.n_steps);
    } while (p.n_steps == 0);
}

// Up to 16 steps of one pair: lane i holds the page and scales of half i (16 tokens).
struct Batch {
    Place p;
    int n;      // steps
    int pg;     // -1: no page
    float ks, vs;
};

__device__ __forceinline__ void load_batch(const AttnArgs &a, const Place &p, int n, Batch &t, bool *bad) {
    const int lane = threadIdx.x & 31;
    t.p = p;
    t.n = n;
    t.pg = -1;
    t.ks = t.vs = 0.f;
    const unsigned tok = (unsigned)p.s * kStep + lane * 16;
    if (tok < (unsigned)p.len && lane < 2 * n) {
        const int pg = a.table[(size_t)p.b * a.table_cap + (tok >> (31 - __clz(a.kc.page)))];
        if ((unsigned)pg < (unsigned)a.kc.n_pages) {
            t.pg = pg;
            t.ks = a.kc.k_scale[(size_t)pg * a.kc.Hkv + p.h];
            t.vs = a.kc.v_scale[(size_t)pg * a.kc.Hkv + p.h];
        } else {
            *bad = true;
        }
    }
}

// The first and the last pair of a team's stretch: number, place of its first
// step on the line, steps, and queries.
struct Stretch {
    int pair[2], x0[2], n[2], nn[2];
};

// Partials (m, l, acc) of one query row put together: acc = sum 2^(m_i - m)
// acc_i, l likewise.  Lane i has channels 4i .. 4i + 3.
struct Merged {
    float m, l;
    float4 acc;
};

__device__ __forceinline__ void add_scaled(float4 &acc, const float4 &v, float w) {
    acc = make_float4(acc.x + v.x * w, acc.y + v.y * w, acc.z + v.z * w, acc.w + v.w * w);
}

// Weights of up to 32 partials, lane i's in lane i (x: its m and l; without any
// seen token every weight is 1, of zeros).  Sets m and l of all of them.
__device__ __forceinline__ float merge_weights(const float2 &x, Merged &r) {
    r.m = x.x;
#pragma unroll
    for (int d = 16; d; d >>= 1) r.m = fmaxf(r.m, __shfl_xor_sync(0xffffffffu, r.m, d));
    const float e = r.m == -INFINITY ? 1.f : exp2_approx(x.x - r.m);
    r.l = x.y * e;
#pragma unroll
    for (int d = 16; d; d >>= 1) r.l += __shfl_xor_sync(0xffffffffu, r.l, d);
    return e;
}

__device__ __forceinline__ void write_row(float *out, const Merged &r) {
    const float f = r.l == 0.f ? 0.f : 1.f / r.l;
    reinterpret_cast<float4 *>(out)[threadIdx.x & 31] =
        make_float4(r.acc.x * f, r.acc.y * f, r.acc.z * f, r.acc.w * f);
}

// kNT: 8-row groups a warp works on; 0: up to 4 rows, whose second copy in
// the group's other 4 places carries P's low halves through the same product.
template <typename E, int kType, int kNT>
__global__ void __launch_bounds__(AtGeom<kNT>::kThreads, 1)
    attn_kv8_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    const E *q, const AttnArgs a) {
    constexpr int kAtWarps = AtGeom<kNT>::kWarps, kAtThreads = AtGeom<kNT>::kThreads;
    constexpr int kN = kNT ? kNT : 1;              // 8-row groups
    constexpr int kRows = kNT ? 8 * kNT : 4;       // query rows of a warp
    constexpr int kQ = sizeof(E) == 4 ? 2 : 1;     // fp16 halves of a query
    // Steps between two flushes of the running sums: 64 products added to each
    // sum (two a step where P's halves share a product, else four).  32 steps in
    // the second case left errors of 1.4e-6 (fp32 sums: 1.3e-6, 16 steps: 7e-7);
    // 12, 16, 24 and 32 steps took 78.1, 76.5, 75.8 and 75.1 us of a verify step.
    constexpr int kFlushSteps = kNT ? 16 : 32;
    extern __shared__ unsigned char sm_raw[];
    __shared__ int before[kAtThreads + 1];   // steps (of one kv head) before each thread's rows
    __shared__ int wsum[kAtThreads / 32];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages];
    __shared__ StageMeta meta[kMaxStages];
    __shared__ Stretch stretch[kMaxTeams];
    __shared__ int last_c0[2], last_c1[2], last_nn[2], last_pair[2];  // pairs that this CTA is the last to finish
    const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in all lanes
    const int tw = a.team_warps, n_teams = kAtWarps / tw, team = warp / tw, wt = warp % tw;
    const int Hkv = a.kc.Hkv, ns = a.n_stages;
    const uint32_t ring = (smem_u32(sm_raw) + 1023u) & ~1023u;

    if (tid < kMaxTeams) stretch[tid].pair[0] = stretch[tid].pair[1] = -1;
    if (tid < kMaxStages) {
        mbar_init(smem_u32(&full[tid]), 1);
        mbar_init(smem_u32(&empty[tid]), tw);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    // what needs no memory, before the wait
    int qi[kN][2];  // which of its head's queries rows 2c, 2c + 1 of each group are (n_q: none)
#pragma unroll
    for (int t = 0; t < kN; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = wt * kRows + (kNT ? t * 8 + 2 * c + j : (2 * c + j) & 3);
            qi[t][j] = row < a.rows ? row % a.n_q : a.n_q;
        }
    const int parts = max(1, kAtWarps / a.rows);  // of the last merge: warps per row
    const int mg_row = warp / parts, mg_part = warp - mg_row * parts;
    const int per = (a.B + kAtThreads - 1) / kAtThreads, n_look = (a.B + per - 1) / max(per, 1);  // rows a thread looks at
    wait_for_prior_kernel();

    // ---- the line: steps before each thread's rows, and in all
    {
        int mine = 0;
        bool bad = false;
#pragma unroll 1
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            if (b < a.B) {
                const int len = clamped_len(a, b), nn = a.n_new ? a.n_new[b] : a.n_q;
                bad |= len != a.lens[b] || nn < 0 || nn > a.n_q;
                mine += steps_of(len);
            }
        }
        if (bad && blockIdx.x == 0) atomicOr(a.ws, kDevBadArg);
        int v = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += y;
        }
        if (lane == 31) wsum[warp] = v;
        __syncthreads();
        int pre = 0;
#pragma unroll 1
        for (int w = 0; w < warp; ++w) pre += wsum[w];
        before[tid + 1] = pre + v;
        if (tid == 0) before[0] = 0;
        __syncthreads();
    }
    const int total = uniform(before[kAtThreads] * Hkv);
    const int cta_share = max((int)(((unsigned)total + gridDim.x - 1) / gridDim.x), kMinCtaSteps);
    const int share = (cta_share + n_teams - 1) / n_teams;
    const int cta_from = (int)min((long long)blockIdx.x * cta_share, (long long)total);
    const int cta_steps = min(cta_share, total - cta_from);
    const int from = (int)((unsigned)cta_from + team * share);  // past the line's end: no steps
    // teams without steps (and warps that make no whole team) only help to merge
    const int steps = team < n_teams ? max(0, min(share, cta_steps - team * share)) : 0;
    const int tm = blockIdx.x * n_teams + team;
    const int st0 = team * ns;
    const uint32_t base = ring + (uint32_t)st0 * kStageBytes;
    // ---- the team's first warp keeps its part of the ring full
    Batch cur = {}, nxt = {};
    Place pl = {};                                   // the first step not yet in a batch
    int to_load = steps, to_issue = steps, in_cur = 0;  // steps in no batch, steps not issued, place in cur
    bool bad = false;
    auto fetch = [&]() {
        nxt.n = 0;
        if (to_load == 0) return;
        if (pl.s == pl.n_steps) next_pair(a, pl);
        const int n = min(min(16, pl.n_steps - pl.s), to_load);
        load_batch(a, pl, n, nxt, &bad);
        pl.s += n;
        to_load -= n;
    };
    auto issue = [&](int st) {  // the next step into stage st
        if (in_cur == cur.n) {
            cur = nxt;
            in_cur = 0;
        }
        const int page = opaque(a.kc.page), tok = (cur.p.s + in_cur) * kStep, len = cur.p.len;
        // lane i < 2: half i
        const int src = (2 * in_cur + (lane & 1)) & 31;
        const int pg = __shfl_sync(0xffffffffu, cur.pg, src);
        const uint32_t bar = smem_u32(&full[st0 + st]), dst = base + (uint32_t)st * kStageBytes;
        const uint32_t have = __ballot_sync(0xffffffffu, pg >= 0) & 3u;
        if (page >= kStep) {
            if (lane == 0 && pg >= 0) {
                const int row = (pg * Hkv + cur.p.h) * page + (tok & (page - 1));
                tma_rows(dst, &map_k, row, bar);
                tma_rows(dst + kStep * kD, &map_v, row, bar);
            }
        } else if (lane < 2 && pg >= 0) {
            const int row = (pg * Hkv + cur.p.h) * 16;
            tma_rows(dst + lane * 16 * kD, &map_k, row, bar);
            tma_rows(dst + (kStep + lane * 16) * kD, &map_v, row, bar);
        }
        // the copies are on their way before the scales are waited for; the
        // barrier cannot complete before its one arrival below
        const float ks = __shfl_sync(0xffffffffu, cur.ks, src), vs = __shfl_sync(0xffffffffu, cur.vs, src);
        StageMeta &m = meta[st0 + st];
        if (lane < 2) {
            m.ks[lane] = ks;
            m.vs[lane] = vs;
            m.nv[lane] = pg >= 0 ? min(16, len - tok - lane * 16) : 0;
        } else if (lane == 2) {
            m.b = cur.p.b;
            m.h = cur.p.h;
            m.s = cur.p.s + in_cur;
            m.n_steps = cur.p.n_steps;
            m.len = len;
        }
        __syncwarp();
        if (lane == 0) mbar_expect_tx(bar, page >= kStep ? (have & 1u) * 2 * kStep * kD : __popc(have) * 2 * 16 * kD);
        // pages and scales of the batch after this one, once this one is under way
        if (in_cur == (cur.n > 1 ? 1 : 0)) fetch();
        ++in_cur;
        --to_issue;
    };
    if (wt == 0 && steps > 0) {  // the step where the team starts
        int lo = 0, hi = n_look;  // the last thread whose rows start at or before it
#pragma unroll 1
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before[mid] * Hkv <= from) lo = mid;
            else hi = mid;
        }
        int pos = from - before[lo] * Hkv;
#pragma unroll 1
        for (int b = lo * per;; ++b) {
            set_row(a, pl, b);
            if (pos < pl.n_steps * Hkv) break;
            pos -= pl.n_steps * Hkv;
        }
        pl.b = uniform(pl.b);
        pl.len = uniform(pl.len);
        pl.n_steps = uniform(pl.n_steps);
        pl.h = uniform(pos / pl.n_steps);
        pl.s = uniform(pos - pl.h * pl.n_steps);
        fetch();
        cur = nxt;
    }

    // ---- all warps of the team consume
    uint32_t qh[kQ][kN][16];      // B fragments of the queries
    float qf[kN][2];              // score factor of rows 2c, 2c + 1
    int lim[kN][2];               // the last token they see
    float o[kN][8][4], m[kN][2], l[kN][2];
    float vs_max = 0.f;           // value scales up to this leave every p <= 2^kSlack in fp16
    float pf[kN][2];              // 2^(6 - E), E: log2 of the row's largest p * value scale; 0: none yet
    int b = -1, h = 0, nn = 0, first_full = 0;
    bool starts_pair = false, ends_pair = false;
    auto begin_pair = [&](const StageMeta &mt) {
        b = mt.b;
        h = mt.h;
        nn = opaque(a.n_new != nullptr) ? min(max(a.n_new[b], 0), a.n_q) : a.n_q;
        first_full = uniform(mt.len - nn + 1);  // tokens below this are seen by every query
        starts_pair = mt.s == 0;
        const E *qb = q + ((size_t)b * Hkv + h) * a.rows * kD;
#pragma unroll
        for (int t = 0; t < kN; ++t) {
            const int r = wt * kRows + (kNT ? t * 8 + g : (g & 3));
            float x[32], top = 0.f;
            if (r < a.rows) {
                const uint4 *src = reinterpret_cast<const uint4 *>(qb + (size_t)r * kD + c * 32);
#pragma unroll
                for (int i = 0; i < (int)sizeof(E) * 2; ++i) {
                    const uint4 u = src[i];
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
                lim[t][j] = qi[t][j] < nn ? mt.len - nn + qi[t][j] : -1;
                m[t][j] = -INFINITY;
                l[t][j] = pf[t][j] = 0.f;
            }
            vs_max = INFINITY;
#pragma unroll
            for (int j = 0; j < 8; ++j) o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.f;
        }
    };
    // The running sums leave the registers: at the end of a pair, and every
    // kFlushSteps steps on the way.  The tensor cores cut off what they add up
    // (towards zero), which over 110 steps grew to 4e-6 of the result and would
    // go on growing; a flush writes the sums to global memory, lane by lane, and
    // starts them at zero, and the next one adds what was written in fp32.
    bool flushed = false;
    auto put_sums = [&](bool last, bool on_the_way) {
        if (flushed || on_the_way) {
            float4 *mine = a.flush + (size_t)(blockIdx.x * kAtWarps + warp) * (9 * kN * 32) + lane;
#pragma unroll
            for (int t = 0; t < kN; ++t, mine += 9 * 32) {
                if (flushed) {
                    float4 v[8];  // all loads before the first use
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = __ldcg(mine + j * 32);
                    const float4 was = __ldcg(mine + 8 * 32);
                    const float k0 = was.x == -INFINITY ? 0.f : exp2_approx(was.x - m[t][0]);
                    const float k1 = was.y == -INFINITY ? 0.f : exp2_approx(was.y - m[t][1]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        o[t][j][0] += v[j].x * k0 * pf[t][0];
                        o[t][j][1] += v[j].y * k1 * pf[t][1];
                        o[t][j][2] += v[j].z * k0 * pf[t][0];
                        o[t][j][3] += v[j].w * k1 * pf[t][1];
                    }
                }
                if (on_the_way) {
                    const float f0 = inverse_pow2(pf[t][0]), f1 = inverse_pow2(pf[t][1]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        __stcg(mine + j * 32,
                               make_float4(o[t][j][0] * f0, o[t][j][1] * f1, o[t][j][2] * f0, o[t][j][3] * f1));
                        o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.f;
                    }
                    __stcg(mine + 8 * 32, make_float4(m[t][0], m[t][1], 0.f, 0.f));
                }
            }
            flushed = on_the_way;
            if (on_the_way) return;
        }
        const long bh = (long)b * Hkv + h;
        const bool whole = starts_pair && ends_pair;
        // A partial of the stretch's last pair goes to the team's own part of
        // the ring, which it has read by now; one of its first pair, with others
        // behind it, to global memory.
        float *part = reinterpret_cast<float *>(sm_raw + (base - smem_u32(sm_raw)));
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
                if ((kNT == 0 && c >= 2) || qi[t][j] >= nn) continue;
                float *dst;
                const float f = inverse_pow2(pf[t][j]);
                float f_l = 1.f;
                if (whole) {
                    dst = a.out + (bh * a.rows + row) * kD;
                    f_l = l[t][j] == 0.f ? 0.f : 1.f / l[t][j];
                } else {
                    const size_t at = last ? (size_t)row : (size_t)(tm + bh) * a.rows + row;
                    dst = (last ? part : a.acc) + at * kD;
                    float *ml = last ? part + a.rows * kD : a.ml;
                    if (g == 0) *reinterpret_cast<float2 *>(ml + at * 2) = make_float2(m[t][j], l[t][j]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float4 *>(dst + g * 16 + i * 4) =
                        make_float4(o[t][2 * i][j] * f_l * f, o[t][2 * i][2 + j] * f_l * f,
                                    o[t][2 * i + 1][j] * f_l * f, o[t][2 * i + 1][2 + j] * f_l * f);
            }
        }
    };

    // One loop fills the ring (it < 0), consumes the steps, and ends the last
    // pair (it == steps): each part of the code stands once, because every CTA
    // fetches all of it (this loop unrolled by hand took 12 us more).
    int st = 0, put = 0;  // stages: next to consume, next to fill
    uint32_t parity = 0;
    bool failed = false;
    int since = 0;  // steps whose sums are in the registers
#pragma unroll 1
    for (int it = steps > 0 ? -ns : 1; it <= steps; ++it) {
        if (it >= 0) {
            StageMeta mt;
            if (it < steps) {
                // a wait that ran out does not leave the loop (lanes would part there):
                // the rest is computed from what the stages hold, and thrown away
                if (!failed) failed = !wait_warp(smem_u32(&full[st0 + st]), parity);
                mt = meta[st0 + st];
            }
            const bool over = it == steps || (!failed && uniform(mt.b != b || mt.h != h));
            if (over || since == kFlushSteps) {
                since = 0;
                if (it == steps && opaque(tw) > 1) asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(tw * 32) : "memory");
                if (uniform(b >= 0) && !failed) put_sums(it == steps, !over);
                if (it == steps) break;
            }
            if (over) {
                begin_pair(mt);
                if (wt == 0 && lane == 0) {  // for the merge
                    const int i = it == 0 ? 0 : 1;
                    stretch[team].pair[i] = stretch[team].pair[1] = b * Hkv + h;
                    stretch[team].x0[i] = stretch[team].x0[1] = from + it - mt.s;
                    stretch[team].n[i] = stretch[team].n[1] = mt.n_steps;
                    stretch[team].nn[i] = stretch[team].nn[1] = nn;
                }
            }
            ++since;
            ends_pair = mt.s + 1 == mt.n_steps;
            const uint32_t kb = base + (uint32_t)st * kStageBytes, vb = kb + kStep * kD;
            const int t0 = uniform(mt.s) * kStep;

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
            const bool holes = uniform(mt.nv[0] < 16 || mt.nv[1] < 16);
            const bool edge = holes || t0 > first_full - kStep;
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
                if (holes) {
#pragma unroll 1
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
                if (kType == SPARK_KV8_E4M3 && opaque(a.n_q) > 1) {
#pragma unroll 1
                    for (int i = max(first_full - t0, 0); i < kStep; ++i) {
                        // (places without a token are zeros by now)
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
            // The reference m of a row's probabilities (a power of two: its log2) is
            // its largest score so far, rounded up, but follows it only when that is
            // more than kSlack above: the sums take any reference, and most steps then
            // need no maximum across lanes and no rescaling.  The same holds for E, the
            // reference of the products p * value scale: it is looked at where m moves,
            // and where a page's value scale alone might bring p out of fp16's range.
            bool move = false;
#pragma unroll
            for (int t = 0; t < kN; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // The scores are rounded here, once: fused into the subtraction below, a
                    // product would lie up to half a step from the m that it gave, which
                    // at scores from 2^27 on brings p out of fp16's range.
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        // above 0, so that an unseen place stays at -inf whatever its page's scale
                        const float f = fmaxf(qf[t][j] * mt.ks[hf], exp2_int(-126));
                        s[t][hf][j] = __fmul_rn(s[t][hf][j], f);
                        s[t][hf][2 + j] = __fmul_rn(s[t][hf][2 + j], f);
                    }
                    const float mx = fmaxf(fmaxf(s[t][0][j], s[t][0][2 + j]), fmaxf(s[t][1][j], s[t][1][2 + j]));
                    move |= mx - m[t][j] > kSlack;  // (m + kSlack may be rounded)
                }
            if (__any_sync(0xffffffffu, move || fmaxf(mt.vs[0], mt.vs[1]) > vs_max)) {
                // value scales are below 2^lv
                const int lv0 = (int)(__float_as_uint(mt.vs[0]) >> 23) - 126;
                const int lv1 = (int)(__float_as_uint(mt.vs[1]) >> 23) - 126;
                float top = 0.f;
#pragma unroll
                for (int t = 0; t < kN; ++t) {
                    float al[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float a0 = fmaxf(s[t][0][j], s[t][0][2 + j]), a1 = fmaxf(s[t][1][j], s[t][1][2 + j]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, d));
                            a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, d));
                        }
                        const float mn = fmaxf(m[t][j], ceilf(fmaxf(a0, a1)));
                        const int up = (int)fminf(mn - m[t][j], 300.f);  // 300 from -inf, and between infinities
                        const bool had = pf[t][j] > 0.f;
                        const int e_old = had ? kPScale + 127 - (int)(__float_as_uint(pf[t][j]) >> 23) - up : -1000;
                        int e = max(e_old, (int)ceilf(fmaxf(a0 - mn + (float)lv0, a1 - mn + (float)lv1)));
                        e = min(max(e, kMinE), kMaxE);
                        const float was = exp2_int(max(-up, -127));  // 0 below 2^-126
                        al[j] = exp2_int(max(e_old - e, -127));
                        l[t][j] *= was;
                        m[t][j] = mn;
                        pf[t][j] = mn == -INFINITY ? 0.f : exp2_int(kPScale - e);
                        top = fmaxf(top, pf[t][j]);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        o[t][j][0] *= al[0];
                        o[t][j][1] *= al[1];
                        o[t][j][2] *= al[0];
                        o[t][j][3] *= al[1];
                    }
                }
                vs_max = kTopFactor * inverse_pow2(top);
            }
            // probabilities, their sums, and the second product
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t ph[kN][2], pl_[kN][2];
#pragma unroll
                for (int t = 0; t < kN; ++t) {
                    const float m0 = m[t][0] == -INFINITY ? 0.f : m[t][0], m1 = m[t][1] == -INFINITY ? 0.f : m[t][1];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float p0 = exp2_approx(s[t][hf][2 * r] - m0);
                        float p1 = exp2_approx(s[t][hf][2 * r + 1] - m1);
                        l[t][0] += p0;
                        l[t][1] += p1;
                        // In this order, as the two factors may be far apart.  Their product kept
                        // finite by a minimum: 140 -> 145 us for 8 rows of 16384 tokens and up to
                        // 32 queries a head (by a bound on pf: 139, but pages then lose bits).
                        p0 = p0 * mt.vs[hf] * pf[t][0];
                        p1 = p1 * mt.vs[hf] * pf[t][1];
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
                }
                if (kType == SPARK_KV8_E4M3 && hide) {
                    __syncwarp();  // a branch, not predicates on the common path
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (t0 + hf * 16 + 2 * c + (i & 1) + (i >> 1) * 8 >= first_full)
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
            __syncwarp();
            if (opaque(tw) > 1 && lane == 0) mbar_arrive(smem_u32(&empty[st0 + st]));
            if (++st == ns) {
                st = 0;
                parity ^= 1;
            }
        }
        // A stage is free once every warp of the team has read it.  A team of
        // one refills it at once; a larger one refills the stage before, which
        // its other warps have most likely left.
        if (opaque(wt) == 0 && to_issue > 0 && !failed && (it != 0 || opaque(tw) == 1)) {
            if (opaque(tw) > 1 && it > 0) {
                // `put` was consumed a step ago, in the lap before this one's unless it has wrapped since
                failed = !wait_warp(smem_u32(&empty[st0 + put]), st > put ? parity : parity ^ 1u);
            }
            if (!failed) issue(put);
            if (++put == ns) put = 0;
        }
    }
    if (failed) {
        if (lane == 0) atomicOr(a.ws, kDevTimeout);
        // let the copies in flight land before the CTA's memory goes away
        if (wt == 0) {
#pragma unroll 1
            for (int i = 0; i < 2 * ns; ++i) wait_warp(smem_u32(&full[st0 + i / 2]), (uint32_t)(i & 1));
        }
    }
    if (bad) atomicOr(a.ws, kDevBadArg);

    // ---- rows without tokens: zeros
#pragma unroll 1
    for (int r = blockIdx.x * kAtWarps + warp; r < a.B; r += gridDim.x * kAtWarps) {
        if (clamped_len(a, r) > 0) continue;
        const int n = a.n_new ? min(max(a.n_new[r], 0), a.n_q) : a.n_q;
        float4 *dst = reinterpret_cast<float4 *>(a.out + (size_t)r * Hkv * a.rows * kD);
#pragma unroll 1
        for (int i = 0; i < Hkv * a.rows; ++i)
            if (i % a.rows % a.n_q < n) dst[(size_t)i * 32 + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    }

    // ---- pairs that several teams share.  Lane t of every warp looks at team
    // t's first and last pair; the first team of this CTA that has steps of a
    // pair stands for it.
    __syncthreads();
    const int cta0 = blockIdx.x * n_teams, cta_to = cta_from + cta_steps;
    bool job[2] = {false, false}, cross[2] = {false, false};
    int pr[2] = {-1, -1}, qn[2] = {0, 0}, x0[2] = {0, 0}, x1[2] = {0, 0};  // the pairs, their queries, first and last step
    if (lane < n_teams && lane * share < cta_steps) {
        const Stretch x = stretch[lane];
        const int f = cta_from + lane * share, t = f + min(share, cta_to - f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            pr[i] = x.pair[i];
            qn[i] = x.nn[i];
            x0[i] = x.x0[i];
            x1[i] = x.x0[i] + x.n[i] - 1;
            job[i] = pr[i] >= 0 && (x0[i] < f || x1[i] >= t);  // others have steps of it
        }
        job[0] = job[0] && (lane == 0 || x0[0] >= f);
        job[1] = job[1] && pr[1] != pr[0];
#pragma unroll
        for (int i = 0; i < 2; ++i) cross[i] = job[i] && (x0[i] < cta_from || x1[i] >= cta_to);
    }
    int c0x[2] = {0, 0}, c1x[2] = {0, 0};  // CTAs that share the pair
    if (warp == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (cross[i]) {
                c0x[i] = x0[i] / cta_share;
                c1x[i] = x1[i] / cta_share;
            }
    }
    int turn = 0;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
#pragma unroll 1
        for (uint32_t todo = __ballot_sync(0xffffffffu, i ? job[1] : job[0]); todo; todo &= todo - 1) {
            const int t = __ffs(todo) - 1;
            const int pair = __shfl_sync(0xffffffffu, i ? pr[1] : pr[0], t);
            // its last team here
            const int te = 31 - __clz(__ballot_sync(0xffffffffu, pr[0] == pair || pr[1] == pair));
            const bool out_too = __shfl_sync(0xffffffffu, (int)!(i ? cross[1] : cross[0]), t) != 0;
            // the last team's partial lies in global memory where other pairs follow in its stretch
            const bool far = __shfl_sync(0xffffffffu, pr[1], te) != pair;
            const int n = __shfl_sync(0xffffffffu, i ? qn[1] : qn[0], t);
#pragma unroll 1
            for (int row = 0, qx = 0; row < a.rows; ++row, ++qx) {
                if (qx == a.n_q) qx = 0;
                if (qx >= n) continue;
                const bool mine = turn == warp;
                if (++turn == kAtWarps) turn = 0;
                if (!mine) continue;
                const size_t at = (size_t)(cta0 + te + pair) * a.rows + row;
                const float *part = reinterpret_cast<const float *>(sm_raw + (ring - smem_u32(sm_raw)));
                const int team_floats = ns * (kStageBytes / 4);
                float4 vf = make_float4(0.f, 0.f, 0.f, 0.f);
                float2 x = make_float2(-INFINITY, 0.f);
                if (far) vf = __ldcg(reinterpret_cast<const float4 *>(a.acc + at * kD) + lane);
                if (lane <= te - t && !(far && lane == te - t))
                    x = *reinterpret_cast<const float2 *>(part + (t + lane) * team_floats + a.rows * kD + row * 2);
                else if (far && lane == te - t)
                    x = __ldcg(reinterpret_cast<const float2 *>(a.ml + at * 2));
                Merged r;
                const float e = merge_weights(x, r);
                r.acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                for (int k = t; k < te + !far; ++k) {
                    const float4 v = reinterpret_cast<const float4 *>(part + k * team_floats + row * kD)[lane];
                    add_scaled(r.acc, v, __shfl_sync(0xffffffffu, e, k - t));
                }
                if (far) add_scaled(r.acc, vf, __shfl_sync(0xffffffffu, e, te - t));
                if (out_too) {
                    write_row(a.out + ((size_t)pair * a.rows + row) * kD, r);
                } else {
                    const size_t to = (size_t)(blockIdx.x + pair) * a.rows + row;
                    __stcg(reinterpret_cast<float4 *>(a.acc_c + to * kD) + lane, r.acc);
                    if (lane == 0) __stcg(reinterpret_cast<float2 *>(a.ml_c + to * 2), make_float2(r.m, r.l));
                }
            }
        }
    }

    // ---- pairs that several CTAs share (at most this CTA's first and last):
    // the last of them to get here merges the CTAs' partials, in their order.
    // A boundary between CTAs lies in one pair, so the first CTA numbers it.
    // (the barrier and the counter's release and acquire order the partials.)
    __syncthreads();
    if (warp == 0) {
        if (lane < 2) last_pair[lane] = -1;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!cross[i]) continue;
            const uint32_t seen = add_acq_rel(a.counter + c0x[i]);
            if (seen == (uint32_t)(c1x[i] - c0x[i])) {
                a.counter[c0x[i]] = 0;  // as the next call needs it
                const int k = c0x[i] < (int)blockIdx.x ? 0 : 1;  // the CTA's first pair, or its last
                last_c0[k] = c0x[i];
                last_c1[k] = c1x[i];
                last_nn[k] = qn[i];
                last_pair[k] = pr[i];
            }
        }
    }
    __syncthreads();
    // one (row, part) a warp where a row has several
    float *sm_acc = reinterpret_cast<float *>(sm_raw), *sm_ml = sm_acc + kAtWarps * kD;
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        const int pair = uniform(last_pair[k]);
        if (pair < 0) continue;
        const int c0 = uniform(last_c0[k]), n = uniform(last_c1[k]) - c0 + 1, each = (n + parts - 1) / parts;
        const int nn_p = uniform(last_nn[k]);
#pragma unroll 1
        for (int row = mg_row; row < a.rows; row += kAtWarps) {
            const int i0 = mg_part * each, i1 = min(n, i0 + each);
            if ((a.n_q > 1 ? row % a.n_q : 0) >= nn_p) continue;
            Merged r = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 1
            for (int i = i0; i < i1; i += 8) {  // 8 at a time, all loads before the weights
                const size_t at = (size_t)(c0 + i + pair) * a.rows + row, step = a.rows;
                const int cnt = min(8, i1 - i);
                float4 v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    v[u] = u < cnt ? __ldcg(reinterpret_cast<const float4 *>(a.acc_c + (at + u * step) * kD) + lane)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
                float2 x = make_float2(-INFINITY, 0.f);
                if (lane < cnt) x = __ldcg(reinterpret_cast<const float2 *>(a.ml_c + (at + lane * step) * 2));
                if (lane == 8) x = make_float2(r.m, r.l);  // what the groups before left
                const float4 old = r.acc;
                const float e = merge_weights(x, r);
                r.acc = make_float4(0.f, 0.f, 0.f, 0.f);
                add_scaled(r.acc, old, __shfl_sync(0xffffffffu, e, 8));
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (u < cnt) add_scaled(r.acc, v[u], __shfl_sync(0xffffffffu, e, u));
            }
            if (parts == 1) {
                write_row(a.out + ((size_t)pair * a.rows + row) * kD, r);
            } else {
                reinterpret_cast<float4 *>(sm_acc + warp * kD)[lane] = r.acc;
                if (lane == 0) reinterpret_cast<float2 *>(sm_ml)[warp] = make_float2(r.m, r.l);
            }
        }
        if (parts == 1) continue;
        __syncthreads();
#pragma unroll 1
        for (int row = warp; row < a.rows; row += kAtWarps) {
            if ((a.n_q > 1 ? row % a.n_q : 0) >= nn_p) continue;
            Merged r;
            const float e = merge_weights(
                lane < parts ? reinterpret_cast<const float2 *>(sm_ml)[row * parts + lane] : make_float2(-INFINITY, 0.f), r);
            r.acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int i = 0; i < parts; ++i)
                add_scaled(r.acc, reinterpret_cast<const float4 *>(sm_acc + (row * parts + i) * kD)[lane],
                           __shfl_sync(0xffffffffu, e, i));
            write_row(a.out + ((size_t)pair * a.rows + row) * kD, r);
        }
        __syncthreads();
    }
}

template <typename E, int kType, int kNT>
static cudaError_t launch_one(const CUtensorMap &mk, const CUtensorMap &mv, const void *q, const AttnArgs &a,
                              int num_sms, cudaStream_t st) {
    const size_t smem = kRingBytes + 1024;
    auto kernel = attn_kv8_kernel<E, kType, kNT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_after_prior(kernel, (unsigned)num_sms, AtGeom<kNT>::kThreads, smem, st, mk, mv,
                              static_cast<const E *>(q), a);
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
    a.counter = reinterpret_cast<uint32_t *>(w + kWsHeader);
    const long pairs = (long)B * kc.Hkv;
    const size_t team_rows = (size_t)attn_team_slots(pairs, num_sms) * a.rows;
    const size_t cta_rows = (size_t)(num_sms + pairs) * a.rows;
    a.flush = reinterpret_cast<float4 *>(w + kWsHeader + attn_counter_bytes(num_sms));
    a.acc = reinterpret_cast<float *>(w + kWsHeader + attn_counter_bytes(num_sms) + num_sms * kFlushBytes);
    a.acc_c = a.acc + team_rows * kD;
    a.ml = a.acc_c + cta_rows * kD;
    a.ml_c = a.ml + team_rows * 2;
    CUtensorMap mk, mv;
    const long rows = (long)kc.n_pages * kc.Hkv * kc.page;
    // a pool without pages is never read: any address does
    if (!make_kv8_map(&mk, rows ? kc.k : ws, rows ? rows : 1, kc.page < kStep ? kc.page : kStep) ||
        !make_kv8_map(&mv, rows ? kc.v : ws, rows ? rows : 1, kc.page < kStep ? kc.page : kStep))
        return cudaErrorInvalidValue;
    const bool e4 = kc.type == SPARK_KV8_E4M3;
    if (dtype == SPARK_F32)
        return e4 ? launch_rows<float, SPARK_KV8_E4M3>(mk, mv, q, a, num_sms, st)
                  : launch_rows<float, SPARK_KV8_I8>(mk, mv, q, a, num_sms, st);
    return e4 ? launch_rows<__nv_bfloat16, SPARK_KV8_E4M3>(mk, mv, q, a, num_sms, st)
              : launch_rows<__nv_bfloat16, SPARK_KV8_I8>(mk, mv, q, a, num_sms, st);
}

}  // namespace spark
