// Write of new keys and values into the paged 8-bit cache (spark_kv8_append).
//
// The scale of a (page, kv head) is 2^E with the smallest E that brings the
// largest |x| of the tokens under the largest code, so scaling is exact and a
// value is rounded once; where a page already holds tokens its E only grows,
// and the old codes are rounded again by a power of two.  One pass: a piece
// of the rows (up to `page` tokens of one head, 4 KB a warp in bf16) stays in
// registers between the maximum and the conversion.  Bound by memory: each
// value is read once and its code written once.
#include "kv8.cuh"

namespace spark {

constexpr int kApWarps = 8;       // warps per CTA
constexpr int kApTokens = 16;     // tokens a warp holds in registers

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

// Warps of one team meet (each team of a CTA has its own barrier).
__device__ __forceinline__ void team_sync(int team, int warps) {
    if (warps == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
}

template <typename E, int kType>
__global__ void __launch_bounds__(kApWarps * 32)
    kv8_append_kernel(const E *__restrict__ k_new, const E *__restrict__ v_new, int B, int n_cap,
                      const int32_t *__restrict__ slots, spark_kv8cache kc, int pieces, uint32_t *status) {
    __shared__ float part[kApWarps];
    constexpr int kVec = 16 / (int)sizeof(E);       // values per 16-byte load
    constexpr int kRowLanes = kD / kVec;            // lanes per token: 16 (bf16) or 32 (fp32)
    constexpr int kPer = 32 / kRowLanes;            // tokens per load instruction
    constexpr int kLoads = kApTokens / kPer;
    const int page = kc.page, Hkv = kc.Hkv;
    const int tw = page / kApTokens;                // warps per team
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int team = warp / tw, wt = warp % tw;
    const long units = (long)B * pieces * Hkv * 2;
    const long unit = (long)blockIdx.x * (kApWarps / tw) + team;
    if (unit >= units) return;
    const bool is_v = (unit & 1) != 0;
    const int h = (int)((unit >> 1) % Hkv);
    const int piece = (int)((unit >> 1) / Hkv % pieces), b = (int)((unit >> 1) / Hkv / pieces);
    const int32_t *row = slots + (size_t)b * n_cap;
    const E *src = (is_v ? v_new : k_new) + ((size_t)b * Hkv + h) * n_cap * kD;
    uint8_t *codes = static_cast<uint8_t *>(is_v ? kc.v : kc.k);
    float *scales = is_v ? kc.v_scale : kc.k_scale;
    const int end = min(n_cap, (piece + 1) * page), n_slots = kc.n_pages * page;
    bool bad = false;
    Run r = next_run(row, piece * page, end, n_cap, page, n_slots, &bad);
    while (r.n > 0) {
        const int o = r.slot & (page - 1);
        const size_t ph = (size_t)(r.slot / page) * Hkv + h;
        uint8_t *dst = codes + ph * page * kD;
        // this warp's tokens of the run: t0 .. t0 + 15
        const int t0 = wt * kApTokens, sub = lane / kRowLanes, col = lane % kRowLanes;
        uint4 x[kLoads];
        const float old = o > 0 ? scales[ph] : 0.f;
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int t = t0 + i * kPer + sub;
            x[i] = t < r.n ? __ldg(reinterpret_cast<const uint4 *>(src + (size_t)(r.j + t) * kD) + col)
                           : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const E *e = reinterpret_cast<const E *>(&x[i]);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const float y = fabsf(Elem<E>::to_f(e[j]));
                a = y < INFINITY ? fmaxf(a, y) : a;  // infinities and NaN do not set the scale
            }
        }
        a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
        if (tw > 1) {
            team_sync(team, tw);  // the last run's maxima have been read
            if (lane == 0) part[warp] = a;
            team_sync(team, tw);
            for (int i = 0; i < tw; ++i) a = fmaxf(a, part[team * tw + i]);
        }
        const int ex = kv8_exponent<kType>(a);
        const float need = exp2_int(ex);
        const bool keeps = o > 0 && old >= need;
        const float inv = keeps ? 1.0f / old : exp2_int(-ex);
        if (o > 0 && !keeps) {  // the page's codes move to the larger scale
            const float ratio = old * inv;
            for (int i = wt * 32 + lane; i < o * (kD / 16); i += tw * 32) {
                uint4 w = *(reinterpret_cast<const uint4 *>(dst) + i);
                uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 lo = __half22float2(kv8_decode2<kType>(u[j] & 0xffffu));
                    const float2 hi = __half22float2(kv8_decode2<kType>(u[j] >> 16));
                    u[j] = kv8_encode2<kType>(lo.x * ratio, lo.y * ratio) |
                           (kv8_encode2<kType>(hi.x * ratio, hi.y * ratio) << 16);
                }
                *(reinterpret_cast<uint4 *>(dst) + i) = w;
            }
        }
        if (wt == 0 && lane == 0 && !keeps) scales[ph] = need;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int t = t0 + i * kPer + sub;
            if (t < r.n) {
                const E *e = reinterpret_cast<const E *>(&x[i]);
                uint32_t c[kVec / 4];
#pragma unroll
                for (int j = 0; j < kVec; j += 4)
                    c[j / 4] = kv8_encode2<kType>(Elem<E>::to_f(e[j]) * inv, Elem<E>::to_f(e[j + 1]) * inv) |
                               (kv8_encode2<kType>(Elem<E>::to_f(e[j + 2]) * inv, Elem<E>::to_f(e[j + 3]) * inv) << 16);
                uint8_t *to = dst + (size_t)(o + t) * kD + col * kVec;
                if (kVec == 8)
                    *reinterpret_cast<uint2 *>(to) = make_uint2(c[0], c[kVec / 4 - 1]);
                else
                    *reinterpret_cast<uint32_t *>(to) = c[0];
            }
        }
        // a later run of this piece may lie in the same page
        __threadfence_block();
        team_sync(team, tw);
        r = next_run(row, r.j + r.n, end, n_cap, page, n_slots, &bad);
    }
    if (bad) atomicOr(status, kDevBadArg);
}

template <typename E>
static cudaError_t launch_append(const E *k_new, const E *v_new, int B, int n_cap, const int32_t *slots,
                                 const spark_kv8cache &kc, void *ws, cudaStream_t st) {
    const int pieces = (n_cap + kc.page - 1) / kc.page;
    const int teams = kApWarps / (kc.page / kApTokens);
    const long units = (long)B * pieces * kc.Hkv * 2;
    const unsigned grid = (unsigned)((units + teams - 1) / teams);
    uint32_t *status = static_cast<uint32_t *>(ws);
    if (kc.type == SPARK_KV8_E4M3)
        kv8_append_kernel<E, SPARK_KV8_E4M3><<<grid, kApWarps * 32, 0, st>>>(k_new, v_new, B, n_cap, slots, kc,
                                                                             pieces, status);
    else
        kv8_append_kernel<E, SPARK_KV8_I8><<<grid, kApWarps * 32, 0, st>>>(k_new, v_new, B, n_cap, slots, kc,
                                                                           pieces, status);
    return cudaGetLastError();
}

cudaError_t launch_kv8_append(const void *k_new, const void *v_new, int B, int n_cap, int dtype,
                              const int32_t *slots, const spark_kv8cache &kc, void *ws, cudaStream_t st) {
    if (dtype == SPARK_F32)
        return launch_append(static_cast<const float *>(k_new), static_cast<const float *>(v_new), B, n_cap, slots, kc,
                             ws, st);
    return launch_append(static_cast<const __nv_bfloat16 *>(k_new), static_cast<const __nv_bfloat16 *>(v_new), B,
                         n_cap, slots, kc, ws, st);
}

}  // namespace spark
