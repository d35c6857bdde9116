// Page tables and slot maps of a paged cache, built on the GPU from request
// lengths (spark_pages_extend), and the return of pages (spark_pages_trim).
//
// With P tokens a page, row b holds have_b = ceil(len_b / P) pages.
//   extend: want_b = ceil((len_b + new_b) / P); its add_b = want_b - have_b new
//           pages are pool[base_b ...], base_b = taken + sum of add over the
//           rows before it.  The slot of token len_b + j is
//           page * P + (len_b + j) mod P.
//   trim:   left_b = ceil(min(keep_b, len_b) / P); the have_b - left_b pages
//           behind it go back to pool[taken - total + (pages of rows before)].
// Both are a prefix sum over the rows and a copy.  Each CTA sums the rows
// before its own itself (a few loads a thread, from L2), which costs less than
// a second launch for the sum at serving batches.  The work grows with B^2, and
// extend's with the 2048-slot pieces of a row too, each a CTA that sums anew:
// one token a row takes 6 us for 512 rows (each without a page before), 14 for
// 4096, 94 for 16384, 1.2 ms for 65536, the most a call takes (trim 5, 15, 163,
// 2.4 ms); 8192 tokens a row 10 us for 512 rows, 71 for 4096 (their slots alone
// 21), 471 for 16384 (82), 5.1 ms for 65536 (329).  lens_out may be lens and taken_out may be
// taken (a replayed graph advances them in place): they are then written by
// the last CTA to finish, when every other one has read them.
//
// Bound by latency: a launch, the lengths, the pages (three dependent reads),
// 2.5 to 3.3 us a call back to back for 64 rows and 4.9 us for 2 M slots (9 MB,
// 1.4 us at the copy rate).
#include "kv8.cuh"

namespace spark {

constexpr int kPgThreads = 256;
constexpr int kPgSlots = 8 * kPgThreads;  // slots of one row per CTA

// Row b's tokens and new tokens, brought into range (bad: something was not).
struct PageRow {
    int len, n_new;
    bool bad;
};

__device__ __forceinline__ PageRow page_row(const int32_t *lens, const int32_t *n_new, int b, int n_cap,
                                            int max_len) {
    const int l = lens[b], n = n_new[b];
    PageRow r;
    r.len = min(max(l, 0), max_len);
    r.n_new = min(min(max(n, 0), n_cap), max_len - r.len);
    r.bad = r.len != l || r.n_new != n;
    return r;
}

__device__ __forceinline__ int pages_of(int tokens, int shift) {
    return (int)(((unsigned)tokens + (1u << shift) - 1u) >> shift);
}

// Sum over the CTA; every thread gets it.
__device__ __forceinline__ int cta_sum(int x, int *sm) {
    x = __reduce_add_sync(0xffffffffu, x);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) sm[warp] = x;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int i = 0; i < kPgThreads / 32; ++i) s += sm[i];
    return s;
}

// Exclusive sum over the CTA's threads; *total gets the whole sum.
__device__ __forceinline__ int cta_scan(int x, int *sm, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int v = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += y;
    }
    __syncthreads();
    if (lane == 31) sm[warp] = v;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kPgThreads / 32; ++i) {
        if (i < warp) before += sm[i];
        all += sm[i];
    }
    *total = all;
    return before + v - x;
}

// True in the CTA that finishes last (all its threads); the ticket is left at
// zero for the next call.
__device__ __forceinline__ bool last_cta(uint32_t *ticket, int *flag) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t t = atomicAdd(ticket, 1u);
        *flag = t == gridDim.x - 1;
        if (*flag) *ticket = 0u;
    }
    __syncthreads();
    return *flag != 0;
}

__global__ void __launch_bounds__(kPgThreads)
    pages_extend_kernel(const int32_t *lens, const int32_t *n_new, int B, int shift,
                        const int32_t *pool, int n_pages, const int32_t *taken, int32_t *table,
                        int table_cap, int n_cap, int32_t *slots, int32_t *lens_out,
                        int32_t *taken_out, int32_t *n_served, int chunks, int in_place, uint32_t *ws) {
    __shared__ int sm[kPgThreads / 32];
    __shared__ int flag;
    const int b = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    const int tid = threadIdx.x;
    const int max_len = table_cap << shift;
    wait_for_prior_kernel();
    const int tk = min(max(*taken, 0), n_pages);
    int before = 0;
    for (int i = tid; i < b; i += kPgThreads) {
        const PageRow r = page_row(lens, n_new, i, n_cap, max_len);
        before += pages_of(r.len + r.n_new, shift) - pages_of(r.len, shift);
    }
    const PageRow r = page_row(lens, n_new, b, n_cap, max_len);
    const int base = tk + cta_sum(before, sm);
    const int have = pages_of(r.len, shift), want = pages_of(r.len + r.n_new, shift);
    const int P = 1 << shift;
    int32_t *row = table + (size_t)b * table_cap;
    bool bad = r.bad || *taken != tk, none = base + (want - have) > n_pages;
    // page number pg of the row: an old one from the table, a new one from the
    // pool; -1 and flagged where that is no page, -1 where the pool has run out
    auto page_at = [&](int pg) -> int {
        const int at = base + (pg - have);
        if (pg >= have && at >= n_pages) return -1;
        const int id = pg < have ? row[pg] : pool[at];
        const bool ok = id >= 0 && id < n_pages;
        bad |= !ok;
        return ok ? id : -1;
    };
    // this CTA's share of the row's new pages
    for (int i = have + chunk * kPgThreads + tid; i < want; i += chunks * kPgThreads) row[i] = page_at(i);
    // slots, four at a time where the row starts on 16 bytes
    const int j0 = chunk * kPgSlots, j1 = min(n_cap, j0 + kPgSlots);
    int32_t *srow = slots + (size_t)b * n_cap;
    auto slot_at = [&](int j, int id) { return j < r.n_new && id >= 0 ? id * P + ((r.len + j) & (P - 1)) : -1; };
    if ((n_cap & 3) == 0) {
        for (int j = j0 + tid * 4; j < j1; j += kPgThreads * 4) {
            int4 s = make_int4(-1, -1, -1, -1);
            if (j < r.n_new) {
                const int p0 = (r.len + j) >> shift, p3 = (r.len + min(j + 3, r.n_new - 1)) >> shift;
                const int a = page_at(p0), c = p3 == p0 ? a : page_at(p3);
                s.x = slot_at(j, a);
                s.y = slot_at(j + 1, (r.len + j + 1) >> shift == p0 ? a : c);
                s.z = slot_at(j + 2, (r.len + j + 2) >> shift == p0 ? a : c);
                s.w = slot_at(j + 3, (r.len + j + 3) >> shift == p0 ? a : c);
            }
            *reinterpret_cast<int4 *>(srow + j) = s;
        }
    } else {
        for (int j = j0 + tid; j < j1; j += kPgThreads)
            srow[j] = j < r.n_new ? slot_at(j, page_at((r.len + j) >> shift)) : -1;
    }
    if (bad) atomicOr(ws, kDevBadArg);
    if (none && tid == 0) atomicOr(ws, kDevNoPages);
    // rows that the pool could not serve end with their last page
    auto finish = [&](const PageRow &x, int i, int at, int want_x, int have_x) {
        const int got = have_x + max(0, min(want_x - have_x, n_pages - at));
        const int end = got < want_x ? max(x.len, min(x.len + x.n_new, got << shift)) : x.len + x.n_new;
        lens_out[i] = end;
        if (n_served) n_served[i] = end - x.len;
    };
    if (!in_place) {
        if (chunk == 0 && tid == 0) {
            finish(r, b, base, want, have);
            if (b == B - 1) *taken_out = min(n_pages, base + (want - have));
        }
        return;
    }
    if (!last_cta(ws + 1, &flag)) return;
    int at = tk;
    for (int i0 = 0; i0 < B; i0 += kPgThreads) {
        const int i = i0 + tid;
        PageRow x = {0, 0, false};
        if (i < B) x = page_row(lens, n_new, i, n_cap, max_len);
        const int h = pages_of(x.len, shift), w = pages_of(x.len + x.n_new, shift);
        int total;
        const int pre = cta_scan(w - h, sm, &total);
        if (i < B) finish(x, i, at + pre, w, h);
        at += total;
    }
    if (tid == 0) *taken_out = min(n_pages, at);
}

__global__ void __launch_bounds__(kPgThreads)
    pages_trim_kernel(const int32_t *lens, const int32_t *keep, int B, int shift, int32_t *pool,
                      int n_pages, const int32_t *taken, const int32_t *table, int table_cap,
                      int32_t *lens_out, int32_t *taken_out, int in_place, uint32_t *ws) {
    __shared__ int sm[kPgThreads / 32];
    __shared__ int flag;
    const int b = blockIdx.x, tid = threadIdx.x;
    const int max_len = table_cap << shift;
    wait_for_prior_kernel();
    const int tk = min(max(*taken, 0), n_pages);
    // len and kept tokens of a row, in range
    auto row_of = [&](int i, bool *bad) {
        const int l = lens[i], k = keep[i];
        const int len = min(max(l, 0), max_len);
        *bad = len != l || k < 0;
        return make_int2(len, min(max(k, 0), len));
    };
    int before = 0, all = 0;
    bool bad = false, x;
    for (int i = tid; i < B; i += kPgThreads) {
        const int2 r = row_of(i, &x);
        const int give = pages_of(r.x, shift) - pages_of(r.y, shift);
        all += give;
        if (i < b) before += give;
    }
    const int total = cta_sum(all, sm);
    const int off = cta_sum(before, sm);
    const int2 r = row_of(b, &bad);
    const int left = pages_of(r.y, shift), give = pages_of(r.x, shift) - left;
    const int to = tk - total + off;  // below 0 only where more pages come back than were taken
    for (int i = tid; i < give; i += kPgThreads) {
        const int id = table[(size_t)b * table_cap + left + i];
        const bool ok = id >= 0 && id < n_pages;
        bad |= !ok;
        if (to + i >= 0) pool[to + i] = ok ? id : -1;
    }
    bad |= *taken != tk || total > tk;
    if (bad) atomicOr(ws, kDevBadArg);
    if (!in_place) {
        if (tid == 0) {
            lens_out[b] = r.y;
            if (b == B - 1) *taken_out = max(0, tk - total);
        }
        return;
    }
    if (!last_cta(ws + 1, &flag)) return;
    for (int i = tid; i < B; i += kPgThreads) lens_out[i] = row_of(i, &x).y;
    if (tid == 0) *taken_out = max(0, tk - total);
}

static int log2_page(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

cudaError_t launch_pages_extend(const int32_t *lens, const int32_t *n_new, int B, int page, const int32_t *pool,
                                int n_pages, const int32_t *taken, int32_t *table, int table_cap, int n_cap,
                                int32_t *slots, int32_t *lens_out, int32_t *taken_out, int32_t *n_served, void *ws,
                                cudaStream_t st) {
    const int chunks = n_cap > kPgSlots ? (n_cap + kPgSlots - 1) / kPgSlots : 1;
    return launch_after_prior(pages_extend_kernel, (unsigned)((long)B * chunks), kPgThreads, 0, st, lens, n_new, B,
                              log2_page(page), pool, n_pages, taken, table, table_cap, n_cap, slots, lens_out,
                              taken_out, n_served, chunks, (int)(lens_out == lens || taken_out == taken),
                              static_cast<uint32_t *>(ws));
}

cudaError_t launch_pages_trim(const int32_t *lens, const int32_t *keep, int B, int page, int32_t *pool, int n_pages,
                              const int32_t *taken, const int32_t *table, int table_cap, int32_t *lens_out,
                              int32_t *taken_out, void *ws, cudaStream_t st) {
    return launch_after_prior(pages_trim_kernel, (unsigned)B, kPgThreads, 0, st, lens, keep, B, log2_page(page), pool,
                              n_pages, taken, table, table_cap, lens_out, taken_out,
                              (int)(lens_out == lens || taken_out == taken), static_cast<uint32_t *>(ws));
}

}  // namespace spark
