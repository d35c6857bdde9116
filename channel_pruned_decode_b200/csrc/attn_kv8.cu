// Attention over the paged 8-bit cache (spark_decode_attn_kv8).
//
// One warp per query row walks the row's tokens: s = q . k * ks / sqrt(D),
// running maximum m and sum l of the softmax, acc = sum p v vs.
#include "kv8.cuh"

namespace spark {

size_t attn_kv8_workspace(int B, int Hkv, int rows, int num_sms) { return kWsHeader; }

template <typename E, int kType>
__global__ void __launch_bounds__(128)
    attn_kv8_kernel(const E *__restrict__ q, spark_kv8cache kc, const int32_t *__restrict__ table, int table_cap,
                    const int32_t *__restrict__ lens, const int32_t *__restrict__ n_new, int B, int G, int n_q,
                    float *__restrict__ out, uint32_t *status) {
    const long r = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long Hq = (long)kc.Hkv * G;
    if (r >= B * Hq * n_q) return;
    const int i = (int)(r % n_q), hq = (int)(r / n_q % Hq), b = (int)(r / n_q / Hq), h = hq / G;
    const int page = kc.page, l0 = lens[b], n0 = n_new ? n_new[b] : n_q;
    const int len = min(max(l0, 0), table_cap * page), nn = min(max(n0, 0), n_q);
    bool bad = len != l0 || nn != n0;
    if (i < nn) {
        const int last = len - nn + i;  // the query's own token
        float qr[4], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
        for (int j = 0; j < 4; ++j) qr[j] = Elem<E>::to_f(q[r * kD + lane * 4 + j]) * 0.08838834764831845f;
        for (int t = 0; t <= last; ++t) {
            const int pg = table[(size_t)b * table_cap + t / page];
            if (pg < 0 || pg >= kc.n_pages) {
                bad = true;
                continue;
            }
            const size_t ph = (size_t)pg * kc.Hkv + h, at = (ph * page + t % page) * kD + lane * 4;
            const uint32_t kw = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(kc.k) + at);
            const uint32_t vw = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(kc.v) + at);
            const float2 k0 = __half22float2(kv8_decode2<kType>(kw & 0xffffu));
            const float2 k1 = __half22float2(kv8_decode2<kType>(kw >> 16));
            float s = (qr[0] * k0.x + qr[1] * k0.y) + (qr[2] * k1.x + qr[3] * k1.y);
            for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            s *= kc.k_scale[ph];
            const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn), pv = p * kc.v_scale[ph];
            const float2 v0 = __half22float2(kv8_decode2<kType>(vw & 0xffffu));
            const float2 v1 = __half22float2(kv8_decode2<kType>(vw >> 16));
            l = l * f + p;
            acc[0] = acc[0] * f + pv * v0.x;
            acc[1] = acc[1] * f + pv * v0.y;
            acc[2] = acc[2] * f + pv * v1.x;
            acc[3] = acc[3] * f + pv * v1.y;
            m = mn;
        }
        for (int j = 0; j < 4; ++j) out[r * kD + lane * 4 + j] = l == 0.f ? 0.f : acc[j] / l;
    }
    if (bad && lane == 0) atomicOr(status, kDevBadArg);
}

cudaError_t launch_attn_kv8(const void *q, int dtype, const spark_kv8cache &kc, const int32_t *table, int table_cap,
                            const int32_t *lens, const int32_t *n_new, int B, int G, int n_q, float *out, void *ws,
                            int num_sms, cudaStream_t st) {
    const long rows = (long)B * kc.Hkv * G * n_q;
    const unsigned grid = (unsigned)((rows + 3) / 4);
    uint32_t *status = static_cast<uint32_t *>(ws);
    auto go = [&](auto kernel, auto *p) {
        kernel<<<grid, 128, 0, st>>>(p, kc, table, table_cap, lens, n_new, B, G, n_q, out, status);
    };
    const float *qf = static_cast<const float *>(q);
    const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(q);
    if (dtype == SPARK_F32)
        kc.type == SPARK_KV8_E4M3 ? go(attn_kv8_kernel<float, SPARK_KV8_E4M3>, qf)
                                  : go(attn_kv8_kernel<float, SPARK_KV8_I8>, qf);
    else
        kc.type == SPARK_KV8_E4M3 ? go(attn_kv8_kernel<__nv_bfloat16, SPARK_KV8_E4M3>, qb)
                                  : go(attn_kv8_kernel<__nv_bfloat16, SPARK_KV8_I8>, qb);
    return cudaGetLastError();
}

}  // namespace spark
