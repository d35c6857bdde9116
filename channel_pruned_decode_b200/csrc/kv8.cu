// Write of new keys and values into the paged 8-bit cache (spark_kv8_append).
//
// The scale of a (page, kv head) is 2^E with the smallest E that brings the
// largest |x| of the tokens under the largest code, so scaling is exact and a
// value is rounded once; where a page already holds tokens its E only grows,
// and the old codes are rounded again by a power of two.  One pass: a piece
// of the rows (up to `page` tokens of one head, 4 KB a warp in bf16) stays in
// registers between the maximum and the conversion.  Bound by memory: each
// value is read once and its code written once (32 rows of 2048 tokens, 8 heads
// in bf16: 63 to 66 us for 378 MB, 88 to 92 % of the copy rate; issue slots
// 60 % used).
#include "kv8.cuh"

namespace spark {

// A warp holds 16 tokens (bf16) or 8 (fp32) in registers, 32 bytes of registers
// a lane and token pair either way; a team of page / tokens warps takes a page.
template <typename E> struct ApGeom {
    static constexpr int kTokens = sizeof(E) == 4 ? 8 : 16;
    static constexpr int kWarps = sizeof(E) == 4 ? 16 : 8;  // per CTA: at least a team of the largest page
};

// A run of tokens that one page takes: the first token and how many.
struct Run {
    int j, n, slot;
};

// The first run that starts in tokens [j, end) of a row of slots, looking at
// 32 tokens at a time; n = 0 if none does.  A run starts where the slot
// before is not the preceding place of the same page.  All lanes agree.
__device__ __forceinline__ Run next_run(const int32_t *row, int j, int end, int n_cap, int page, int n_slots,
                                        bool *bad) {
    const int lane = threadIdx.x & 31;
    Run r = {end, 0, 0};
    for (; j < end; j += 32) {
        const int i = j + lane;
        bool start = false;
        if (i < end) {
            const int s = row[i];
            const bool ok = s >= 0 && s < n_slots;
            *bad |= s >= n_slots;
            start = ok && !(i > 0 && (s & (page - 1)) != 0 && row[i - 1] == s - 1);
        }
        const uint32_t m = __ballot_sync(0xffffffffu, start);
        if (m) {
            r.j = j + __ffs(m) - 1;
            break;
        }
    }
    if (r.j >= end) return r;
    r.slot = row[r.j];
    const int most = min(page - (r.slot & (page - 1)), n_cap - r.j);
    r.n = most;
    for (int i0 = 0; i0 < most; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t off = __ballot_sync(0xffffffffu, i < most && row[r.j + i] != r.slot + i);
        if (off) {
            r.n = i0 + __ffs(off) - 1;
            break;
        }
    }
    return r;
}

// The run of a piece of a row whose slots follow one another from the row's
// first slot on, as spark_pages_extend writes them: tokens [j, end) lie in one
// page, and negative slots may follow.  False: they do not (any other map).
__device__ __forceinline__ bool plain_run(const int32_t *row, int j, int end, int page, int n_slots, int place, Run &r) {
    const int lane = threadIdx.x & 31;
    r = {j, 0, 0};
    bool plain = true, open = true;  // open: no slot has broken off yet
#pragma unroll 1
    for (int i0 = 0; i0 < end - j; i0 += 32) {
        const int i = i0 + lane;
        const int s = j + i < end ? row[j + i] : -1;
        if (i0 == 0) r.slot = __shfl_sync(0xffffffffu, s, 0);
        const uint32_t off = __ballot_sync(0xffffffffu, s < 0 || s != r.slot + i);
        const uint32_t used = __ballot_sync(0xffffffffu, s >= 0);
        const int k = open ? (off ? __ffs(off) - 1 : 32) : 0;
        r.n += k;
        open = open && off == 0;
        plain = plain && (k == 32 || (used >> k) == 0);
    }
    return plain && (r.n == 0 || (r.slot < n_slots && (r.slot & (page - 1)) == place));
}

// Warps of one team meet (each team of a CTA has its own barrier).
__device__ __forceinline__ void team_sync(int team, int warps) {
    if (warps == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
}

// Largest |x| of the loaded values, infinities and NaN left out.  On the bits:
// without the sign they order like the numbers, with infinities and NaN on top.
template <typename E, int kLoads>
__device__ __forceinline__ float largest(const uint4 (&x)[kLoads], bool *special) {
    constexpr bool kWide = sizeof(E) == 4;
    constexpr uint32_t kSign = kWide ? 0x7fffffffu : 0x7fff7fffu, kInf = kWide ? 0x7f800000u : 0x7f80u;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = (&x[i].x)[j] & kSign;
            m = kWide ? max(m, w) : __vmaxu2(m, w);
        }
    if (!kWide) m = max(m & 0xffffu, m >> 16);
    m = __reduce_max_sync(0xffffffffu, m);
    *special = m >= kInf;
    if (*special) {  // once more, without them
        m = 0;
#pragma unroll 1
        for (int i = 0; i < kLoads; ++i) {
            uint4 v = x[0];
#pragma unroll
            for (int u = 1; u < kLoads; ++u)
                if (u == i) v = x[u];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w = (&v.x)[j] & kSign;
                if (kWide) {
                    m = w < kInf ? max(m, w) : m;
                } else {
                    if ((w & 0xffffu) < kInf) m = max(m, w & 0xffffu);
                    if ((w >> 16) < kInf) m = max(m, w >> 16);
                }
            }
        }
        m = __reduce_max_sync(0xffffffffu, m);
    }
    return __uint_as_float(kWide ? m : m << 16);
}

template <typename E> __device__ __forceinline__ void unpack4(const uint4 &x, int half, float (&f)[4]) {
    if (sizeof(E) == 4) {
        f[0] = __uint_as_float(x.x);
        f[1] = __uint_as_float(x.y);
        f[2] = __uint_as_float(x.z);
        f[3] = __uint_as_float(x.w);
    } else {
        const uint32_t a = half ? x.z : x.x, b = half ? x.w : x.y;
        f[0] = __uint_as_float(a << 16);
        f[1] = __uint_as_float(a & 0xffff0000u);
        f[2] = __uint_as_float(b << 16);
        f[3] = __uint_as_float(b & 0xffff0000u);
    }
}

// Codes of four values.  int8 without special values: adding 1.5 * 2^23 rounds
// to a whole number (to even at ties) and leaves it in the low byte.
template <int kType> __device__ __forceinline__ uint32_t encode4(const float (&f)[4], float inv, bool special) {
    if (kType == SPARK_KV8_I8 && !special) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(fmaf(f[i], inv, 12582912.f));
        return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
    }
    const uint16_t lo = (uint16_t)kv8_encode2<kType>(f[0] * inv, f[1] * inv);
    const uint16_t hi = (uint16_t)kv8_encode2<kType>(f[2] * inv, f[3] * inv);
    uint32_t r;
    asm("mov.b32 %0, {%1, %2};" : "=r"(r) : "h"(lo), "h"(hi));
    return r;
}

// 4 CTAs of 8 warps (2 of 16) on an SM: the chain slots -> values -> codes is
// hidden by 32 warps with 4 KB under way each, not inside one.
template <typename E, int kType>
__global__ void __launch_bounds__(ApGeom<E>::kWarps * 32, 32 / ApGeom<E>::kWarps)
    kv8_append_kernel(const E *k_new, const E *v_new, int B, int n_cap, const int32_t *slots,
                      spark_kv8cache kc, int pieces, int per, uint32_t *status) {
    constexpr int kWarps = ApGeom<E>::kWarps, kTokens = ApGeom<E>::kTokens;
    __shared__ float part[kWarps];
    constexpr int kVec = 16 / (int)sizeof(E);       // values per 16-byte load
    constexpr int kRowLanes = kD / kVec;            // lanes per token: 16 (bf16) or 32 (fp32)
    constexpr int kPer = 32 / kRowLanes;            // tokens per load instruction
    constexpr int kLoads = kTokens / kPer;          // 8
    const int page = kc.page, Hkv = kc.Hkv;
    const int tw = page / kTokens;                  // warps per team
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int team = warp / tw, wt = warp - team * tw;
    // a team's work: `per` of the 2 * Hkv (head, key or value)s of one piece of one row
    const unsigned shares = (unsigned)(2 * Hkv + per - 1) / (unsigned)per;
    const unsigned unit = blockIdx.x * (unsigned)(kWarps / tw) + (unsigned)team;
    const unsigned bp = unit / shares, b = bp / (unsigned)pieces;
    if (b >= (unsigned)B) return;
    const int piece = (int)(bp - b * (unsigned)pieces), first = (int)(unit - bp * shares) * per;
    const int last = min(first + per, 2 * Hkv);
    const int32_t *row = slots + (size_t)b * n_cap;
    const int n_slots = kc.n_pages * page;
    wait_for_prior_kernel();
    // a piece is what falls into one page if the row's slots follow one another
    const int o0 = max(row[0], 0) & (page - 1);
    const int begin = max(0, piece * page - o0), end = min(n_cap, (piece + 1) * page - o0);
    if (begin >= end) return;
    bool bad = false;
    Run run;
    const bool plain = plain_run(row, begin, end, page, n_slots, (begin + o0) & (page - 1), run);
    if (!plain) run = next_run(row, begin, end, n_cap, page, n_slots, &bad);
    if (run.n == 0) {
        if (bad) atomicOr(status, kDevBadArg);
        return;
    }
#pragma unroll 1
    for (int w = first; w < last; ++w) {
        const int h = w >> 1;
        const E *src = ((w & 1) ? v_new : k_new) + ((size_t)b * Hkv + h) * n_cap * kD;
        uint8_t *codes = static_cast<uint8_t *>((w & 1) ? kc.v : kc.k);
        float *scales = (w & 1) ? kc.v_scale : kc.k_scale;
        Run r = run;
#pragma unroll 1
        while (r.n > 0) {
            const int o = r.slot & (page - 1);
            const size_t ph = (size_t)(r.slot / page) * Hkv + h;
            uint8_t *dst = codes + ph * page * kD;
            // this warp's tokens of the run: t0 ..
            const int t0 = wt * kTokens, sub = lane / kRowLanes, col = lane % kRowLanes;
            const bool whole = t0 + kTokens <= r.n;  // all of this warp's tokens are there
            uint4 x[kLoads];
            const float old = o > 0 ? scales[ph] : 0.f;
            const uint4 *from = reinterpret_cast<const uint4 *>(src + (size_t)(r.j + t0 + sub) * kD) + col;
            if (whole) {
#pragma unroll
                for (int i = 0; i < kLoads; ++i) x[i] = __ldcs(from + i * kPer * (kD / kVec));
            } else {
#pragma unroll
                for (int i = 0; i < kLoads; ++i)
                    x[i] = t0 + i * kPer + sub < r.n ? __ldcs(from + i * kPer * (kD / kVec)) : make_uint4(0, 0, 0, 0);
            }
            bool special;
            float a = largest<E, kLoads>(x, &special);
            if (tw > 1) {
                team_sync(team, tw);  // the last run's maxima have been read
                if (lane == 0) part[warp] = a;
                team_sync(team, tw);
                a = lane < tw ? part[team * tw + lane] : 0.f;
                a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
            }
            const int ex = kv8_exponent<kType>(a);
            const float need = exp2_int(ex);
            special |= ex == kKv8MaxExp;  // values may lie beyond the largest code
            const bool keeps = o > 0 && old >= need;
            const float inv = keeps ? 1.0f / old : exp2_int(-ex);
            if (o > 0 && !keeps) {  // the page's codes move to the larger scale
                const float ratio = old * inv;
#pragma unroll 1
                for (int i = wt * 32 + lane; i < o * (kD / 16); i += tw * 32) {
                    uint4 w = *(reinterpret_cast<const uint4 *>(dst) + i);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t &c = (&w.x)[j];
                        const float2 lo = __half22float2(kv8_decode2<kType>(c & 0xffffu));
                        const float2 hi = __half22float2(kv8_decode2<kType>(c >> 16));
                        c = kv8_encode2<kType>(lo.x * ratio, lo.y * ratio) |
                            (kv8_encode2<kType>(hi.x * ratio, hi.y * ratio) << 16);
                    }
                    *(reinterpret_cast<uint4 *>(dst) + i) = w;
                }
            }
            if (wt == 0 && lane == 0 && !keeps) scales[ph] = need;
            uint8_t *to = dst + (size_t)(o + t0 + sub) * kD + col * kVec;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                uint32_t c[kVec / 4];
#pragma unroll
                for (int j = 0; j < kVec / 4; ++j) {
                    float f[4];
                    unpack4<E>(x[i], j, f);
                    c[j] = encode4<kType>(f, inv, special);
                }
                if (whole || t0 + i * kPer + sub < r.n) {
                    if (kVec == 8)
                        *reinterpret_cast<uint2 *>(to + i * kPer * kD) = make_uint2(c[0], c[kVec / 4 - 1]);
                    else
                        *reinterpret_cast<uint32_t *>(to + i * kPer * kD) = c[0];
                }
            }
            if (plain) break;
            // a later run of this piece may lie in the same page
            __threadfence_block();
            team_sync(team, tw);
            r = next_run(row, r.j + r.n, end, n_cap, page, n_slots, &bad);
        }
    }
    if (bad) atomicOr(status, kDevBadArg);
}

template <typename E>
static cudaError_t launch_append(const E *k_new, const E *v_new, int B, int n_cap, const int32_t *slots,
                                 const spark_kv8cache &kc, void *ws, int num_sms, cudaStream_t st) {
    constexpr int kWarps = ApGeom<E>::kWarps;
    const int pieces = (n_cap + kc.page - 2) / kc.page + 1;  // a row may start on a page's last place
    const int teams = kWarps / (kc.page / ApGeom<E>::kTokens);
    // Where the GPU is full more than once, a team takes the keys and the values
    // of a head, which share its look at the slots.  32 x
    // 2048 tokens of 8 heads in bf16: 1 at a time 68.7 us, 2 63.0, 4 66.0, 8 67.5,
    // 16 72.3; 5 x 1777 tokens of 4 heads in fp32: 11.4, 9.6, 14.5, 23.5 (the GPU
    // no longer full).
    const long warps = (long)B * pieces * kc.Hkv * 2 * (kWarps / teams);
    const int per = warps > 32l * num_sms ? 2 : 1;
    const long units = (long)B * pieces * ((2 * kc.Hkv + per - 1) / per);
    const unsigned grid = (unsigned)((units + teams - 1) / teams);
    uint32_t *status = static_cast<uint32_t *>(ws);
    auto kernel = kc.type == SPARK_KV8_E4M3 ? kv8_append_kernel<E, SPARK_KV8_E4M3> : kv8_append_kernel<E, SPARK_KV8_I8>;
    return launch_after_prior(kernel, grid, kWarps * 32, 0, st, k_new, v_new, B, n_cap, slots, kc, pieces, per, status);
}

cudaError_t launch_kv8_append(const void *k_new, const void *v_new, int B, int n_cap, int dtype,
                              const int32_t *slots, const spark_kv8cache &kc, void *ws, int num_sms, cudaStream_t st) {
    if (dtype == SPARK_F32)
        return launch_append(static_cast<const float *>(k_new), static_cast<const float *>(v_new), B, n_cap, slots, kc,
                             ws, num_sms, st);
    return launch_append(static_cast<const __nv_bfloat16 *>(k_new), static_cast<const __nv_bfloat16 *>(v_new), B,
                         n_cap, slots, kc, ws, num_sms, st);
}

}  // namespace spark
