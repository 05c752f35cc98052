// kvcache.hip -- writing a paged key-value cache: new tokens' rows into their
// sequences' pages, and the copy of an eviction's kept rows into new pages.
// Both move rows of 16-byte chunks and nothing else: bound by the bytes read
// and written.  16384 tokens of eight 128-wide heads: 28.8 us (134 MB, 4.7
// TB/s); 262144 kept rows of 512 bytes (268 MB) 61 us, 4.4 TB/s; a device copy
// moves 4.9.
#include "device_common.h"
#include "kernels.h"

namespace coli {

constexpr int KVC_NT = 256;
// Most workgroups of an append's launch: 2^30 threads, a launch holds fewer
// than 2^32.  More new tokens (2^22 of the widest are 8 GB and up) take
// several launches.
constexpr int KVC_MAX_WG = 1 << 22;

// Pool row of position p of cache head h, -1 where the page id is none.
__device__ __forceinline__ int pool_row(const int32_t *__restrict__ table_row, int p, int h, int Hkv, int page_shift,
                                        int n_pages)
{
    const int pg = table_row[p >> page_shift];
    if (pg < 0 || pg >= n_pages) return -1;
    return (int)((((uint32_t)pg * (uint32_t)Hkv + (uint32_t)h) << page_shift) +
                 (uint32_t)(p & ((1 << page_shift) - 1)));
}

// One new token a workgroup, or several narrow ones (a.tokens), so that its threads have a chunk each: with
// one, 16384 tokens of two 64-wide heads (32 chunks) took 15.8 us, with
// eight 6.9.  (With one the place is looked up in scalar registers: 16384
// tokens of eight 128-wide heads 28.8 us, 41.9 without.)  The sequence of row r is the last b with start[b] <= r (found by
// halving; start ascends), its position lens[b] - (start[b + 1] - r).
template <bool ONE>
__global__ __launch_bounds__(KVC_NT) void kv_append_kernel(AppendLaunch a)
{
    const int per = a.k_chunks + a.v_chunks, width = a.Hkv * per;
    const int x = ONE ? 0 : (int)threadIdx.x / width;
    const int r = a.first + (ONE ? blockIdx.x : blockIdx.x * a.tokens + x);
    if (!ONE && (x >= a.tokens || r >= a.rows)) return;
    int b = r, p;
    if (a.start) {
        if (r < a.start[0] || r >= a.start[a.B]) return;
        int lo = 0, hi = a.B;                         // start[lo] <= r < start[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.start[mid] <= r) lo = mid;
            else hi = mid;
        }
        b = lo;
        p = min(max(a.lens[b], 0), a.cap) - a.start[b + 1] + r;
    } else {
        p = min(max(a.lens[b], 0), a.cap) - 1;
    }
    if (p < 0 || p >= a.cap) return;
    const int32_t *table = a.table + (size_t)b * a.max_pages;
    const int first = pool_row(table, p, 0, a.Hkv, a.page_shift, a.n_pages);
    if (first < 0) return;
    const uint32_t page = 1u << a.page_shift;
    const u32x4 *__restrict__ k_new = (const u32x4 *)a.k_new, *__restrict__ v_new = (const u32x4 *)a.v_new;
    u32x4 *__restrict__ k = (u32x4 *)a.k, *__restrict__ v = (u32x4 *)a.v;
    for (int i = threadIdx.x - x * width; i < width; i += KVC_NT) {
        const int h = i / per, c = i - h * per, cv = c - a.k_chunks;
        const size_t from = (size_t)r * a.Hkv + h, to = (size_t)((uint32_t)first + (uint32_t)h * page);
        if (cv < 0) k[to * a.k_chunks + c] = k_new[from * a.k_chunks + c];
        else v[to * a.v_chunks + cv] = v_new[from * a.v_chunks + cv];
    }
}

hipError_t launch_kv_append(const AppendLaunch &in, hipStream_t st)
{
    if (in.rows == 0 || in.B == 0) return hipSuccess;
    AppendLaunch a = in;
    const int width = a.Hkv * (a.k_chunks + a.v_chunks);
    a.tokens = width < KVC_NT ? KVC_NT / width : 1;
    const int all = (a.rows + a.tokens - 1) / a.tokens;       // workgroups
    for (int at = 0; at < all; at += KVC_MAX_WG) {
        const int n = min(all - at, KVC_MAX_WG);
        a.first = at * a.tokens;
        if (a.tokens == 1) kv_append_kernel<true><<<n, KVC_NT, 0, st>>>(a);
        else kv_append_kernel<false><<<n, KVC_NT, 0, st>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// The kept rows of one (sequence, cache head), `each` a workgroup: their old
// and new pool rows go through LDS once, then the chunks of all of them are
// copied side by side.  The same workgroups write the kept weights, the zeros
// behind them and the new length.
constexpr int EV_ROWS = 64;              // most rows of a workgroup

__global__ __launch_bounds__(KVC_NT) void kv_evict_copy_kernel(EvictLaunch a, int blocks, int each)
{
    __shared__ int32_t from[EV_ROWS], to[EV_ROWS];
    const int tid = threadIdx.x;
    const int bh = blockIdx.x / blocks, blk = blockIdx.x % blocks;
    const int b = bh / a.Hkv, h = bh % a.Hkv;
    const int n = min(max(a.lens[b], 0), a.cap), m = min(n, a.keep);
    const int j0 = blk * each;
    if (blk == 0 && h == 0 && tid == 0) a.new_lens[b] = m;
    if (tid < each && j0 + tid < max((long)m, a.new_acc ? a.new_ld : 0)) {
        const int j = j0 + tid;
        float w = 0.f;
        if (j < m) {
            const int p = a.kept[(size_t)bh * a.keep + j];
            from[tid] = pool_row(a.table + (size_t)b * a.max_pages, p, h, a.Hkv, a.page_shift, a.n_pages);
            to[tid] = pool_row(a.new_table + (size_t)b * a.new_max_pages, j, h, a.Hkv, a.page_shift, a.n_pages);
            w = a.acc[(size_t)bh * a.ld + p];
        }
        if (a.new_acc && j < a.new_ld) a.new_acc[(size_t)bh * a.new_ld + j] = w;
    }
    __syncthreads();
    // (eight chunks of a thread read before the first is written: 63 against 61 us for 268 MB)
    const int rows = min(each, m - j0);
    u32x4 *k = (u32x4 *)a.k, *v = (u32x4 *)a.v;
    for (int i = tid; i < rows * a.k_chunks; i += KVC_NT) {
        const int r = i / a.k_chunks, c = i - r * a.k_chunks;
        if (from[r] >= 0 && to[r] >= 0) k[(size_t)to[r] * a.k_chunks + c] = k[(size_t)from[r] * a.k_chunks + c];
    }
    for (int i = tid; i < rows * a.v_chunks; i += KVC_NT) {
        const int r = i / a.v_chunks, c = i - r * a.v_chunks;
        if (from[r] >= 0 && to[r] >= 0) v[(size_t)to[r] * a.v_chunks + c] = v[(size_t)from[r] * a.v_chunks + c];
    }
}

hipError_t launch_kv_evict(const EvictLaunch &a, hipStream_t st)
{
    if (a.B == 0) return hipSuccess;
    const hipError_t e =
        launch_index_topk(a.acc, a.B * a.Hkv, a.cap, a.ld, a.lens, a.Hkv, a.keep, a.tail, a.kept, st);
    if (e != hipSuccess) return e;
    const long span = a.new_acc && a.new_ld > a.keep ? a.new_ld : a.keep;
    // Few rows go over more workgroups (us with 16 / 64 rows each, selection
    // included: 2048 rows of 32 chunks in all 10.3 / 12.0, 4001 of 72 chunks
    // 24.1 / 29.9, 65536 of 32 chunks 26.5 / 25.1, 262144 of them 64.6 / 55.3).
    const int each = (long)a.B * a.Hkv * span < (1 << 15) ? 16 : EV_ROWS;
    const int blocks = (int)((span + each - 1) / each);
    kv_evict_copy_kernel<<<a.B * a.Hkv * blocks, KVC_NT, 0, st>>>(a, blocks, each);
    return hipGetLastError();
}

}  // namespace coli
