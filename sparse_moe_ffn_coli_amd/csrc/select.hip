// select.hip -- index selection of the sparse attention's IndexPool: per
// row, the k positions with the largest indexer scores, with the last `tail`
// positions always kept ("Add GLM-5.3-Flash (glm5next) support with ROCmFP
// mix qtypes (105/106)", section "MLA/DSA": top-k over the indexer scores
// with k = 2048, the last kpool tokens always selected).
//
// One workgroup of 16 waves per row.  Scores become order-preserving
// unsigned keys (-0 folded onto +0; the tail positions take the largest key),
// so "larger score first, lower position on ties" is "larger key first,
// lower position on ties".  The k-th largest key tau is found by a radix
// select over three digits (bits 31-21, 20-10, 9-0): an LDS histogram of the
// current digit among the keys that match the digits found so far, and a
// workgroup suffix scan over the bins to find the digit holding the k-th key.
// Every position whose key is above tau is selected, and of those equal to
// tau the lowest positions until k are reached.  The selected positions are
// written in ascending order by an ordered compaction: each thread marks its
// neighbouring positions above and equal to tau in bit masks, and one scan of
// their counts over the workgroup gives it its first slot.  Integer work only:
// the result is unique and reproducible.
// Rows of up to SEL_CAP positions keep their keys in LDS after one read of
// the scores; longer rows re-read the scores (from L2) in each pass.
// Bound by a row's chain of passes and barriers, not by its bytes: 64 rows of
// 32768 scores 16.3 us (8.9 MB), 2048 of them 126 us (277 MB, 2.2 TB/s), one
// row of 131072 71 us.  Neither the next row's scores prefetched into
// registers meanwhile (132 us) nor keys held in registers, two rows a CU
// (143), was faster.
#include "device_common.h"
#include "kernels.h"

namespace coli {

constexpr int SEL_NT = 1024;             // threads per workgroup (16 waves)
constexpr int SEL_WAVES = SEL_NT / 64;
constexpr int SEL_GROUPS = 4;            // groups of four scores a thread of a long row has in flight

// A tail position's key, above every score's: the last NaN's own key would be
// the same and is one less.
constexpr uint32_t TAIL_KEY = 0xffffffffu;

__device__ __forceinline__ uint32_t score_key(float f)
{
    const uint32_t u = __float_as_uint(f);
    uint32_t key = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    key += key == 0x7fffffffu;           // -0 ranks with +0
    return min(key, TAIL_KEY - 1);
}

constexpr int SEL_CAP = 32768;           // positions whose keys a workgroup keeps in LDS (128 KB)
constexpr int SEL_SHORT = 16384;         // the same where no row is longer: two workgroups a CU

// Barrier for LDS traffic only: every wave's LDS operations have completed
// (global loads and stores in flight are not waited for).
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_s_waitcnt(0xc07f);           // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
}

// Inclusive prefix sum over the workgroup in thread order (ws: SEL_WAVES ints).
__device__ __forceinline__ int block_scan_incl_dpp(int v, int32_t *ws)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = wave_scan_incl(v);
    if (lane == 63) ws[wave] = v;
    lds_barrier();
    int before = 0;
#pragma unroll
    for (int w2 = 0; w2 < SEL_WAVES; ++w2) before += (w2 < wave) ? ws[w2] : 0;
    return v + before;
}

// ---- a cached row (n <= 4 SEL_NT PER): keys in LDS, thread t loading the
// groups of four positions 4 (j * SEL_NT + t) .. + 3 ------------------------

// The scores of a row into registers (one 16-byte load per group; the groups
// past the last whole one reread it, their values unused).
template <int PER>
__device__ __forceinline__ void load_row(const float *__restrict__ row, int n, f32x4 (&v)[PER])
{
    const int n4 = n & ~3;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = 4 * (j * SEL_NT + (int)threadIdx.x);
        v[j] = (n4 >= 4) ? *reinterpret_cast<const f32x4 *>(row + min(i, n4 - 4)) : f32x4{0.f, 0.f, 0.f, 0.f};
    }
}

// keys[i] = key of position i, hist[d] = positions whose top 11 key bits are d
template <int PER>
__device__ __forceinline__ void store_keys(const float *__restrict__ row, int n, int tail0, const f32x4 (&v)[PER],
                                           uint32_t *keys, int32_t *hist)
{
    const int n4 = n & ~3;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = 4 * (j * SEL_NT + (int)threadIdx.x);
        if (i < n4) {
            uint32_t q[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                q[c] = (i + c >= tail0) ? TAIL_KEY : score_key(v[j][c]);
                atomicAdd(&hist[q[c] >> 21], 1);
            }
            *reinterpret_cast<u32x4 *>(keys + i) = u32x4{q[0], q[1], q[2], q[3]};
        }
    }
    for (int i = n4 + (int)threadIdx.x; i < n; i += SEL_NT) {     // the last 0-3 positions
        const uint32_t q = (i >= tail0) ? TAIL_KEY : score_key(row[i]);
        keys[i] = q;
        atomicAdd(&hist[q >> 21], 1);
    }
    // up to the next whole 4 * SEL_NT positions: keys that are never selected (compact_cached)
    const int whole = (n + 4 * SEL_NT - 1) / (4 * SEL_NT) * (4 * SEL_NT);
    for (int i = n + (int)threadIdx.x; i < whole; i += SEL_NT) keys[i] = 0u;
}

// The digit holding the need-th largest key: thread t holds bins nb-1-2t and
// nb-2-2t, so a scan in thread order is a suffix scan over the bins.  Returns
// the bin; *above receives the keys in higher bins.  Clears hist afterwards.
__device__ __forceinline__ int pick_bin(int32_t *hist, int nb, int need, int32_t *ws, int32_t *sel_s, int *above_out)
{
    const int tid = threadIdx.x;
    const int b0 = nb - 1 - 2 * tid, b1 = b0 - 1;
    const int c0 = (b0 >= 0) ? hist[b0] : 0, c1 = (b1 >= 0) ? hist[b1] : 0;
    const int incl = block_scan_incl_dpp(c0 + c1, ws);
    const int above = incl - c0 - c1;
    if (above < need && above + c0 >= need) {
        sel_s[0] = b0;
        sel_s[1] = above;
    } else if (above + c0 < need && above + c0 + c1 >= need) {
        sel_s[0] = b1;
        sel_s[1] = above + c0;
    }
    if (b0 >= 0) hist[b0] = 0;                    // every bin is read above by its owner only
    if (b1 >= 0) hist[b1] = 0;
    for (int b = nb + tid; b < 2048; b += SEL_NT) hist[b] = 0;
    lds_barrier();
    const int bin = sel_s[0];
    *above_out = sel_s[1];
    lds_barrier();                                // sel_s and ws are free again
    return bin;
}

// Places a thread's selected positions among the workgroup's: bit i of gt, eq:
// position first + i is above, equal to tau; gt_b, eq_b: such keys before the
// workgroup's first (moved on past its last).
__device__ __forceinline__ void place_masks(uint32_t gt, uint32_t eq, int first, int k, int need, int &gt_b, int &eq_b,
                                            int32_t *ws, int32_t *out)
{
    // at most SEL_CAP positions at a time: both counts fit in 16 bits
    const uint32_t mine = (uint32_t)__popc(gt) | (uint32_t)__popc(eq) << 16;
    const uint32_t before = (uint32_t)block_scan_incl_dpp((int)mine, ws) - mine;
    uint32_t all = 0;
#pragma unroll
    for (int w = 0; w < SEL_WAVES; ++w) all += (uint32_t)ws[w];
    const int my_gt = gt_b + (int)(before & 0xffffu), my_eq = eq_b + (int)(before >> 16);
    gt_b += (int)(all & 0xffffu);
    eq_b += (int)(all >> 16);
    int slot = my_gt + min(my_eq, need);
    const int keep = min(max(need - my_eq, 0), __popc(eq));
    if (keep == 0) eq = 0u;
    for (int drop = __popc(eq) - keep; drop > 0; --drop)      // of equal keys the lowest positions stay
        eq &= ~(0x80000000u >> __clz((int)eq));
    for (uint32_t sel = gt | eq; sel; sel &= sel - 1, ++slot)
        if (slot < k) out[slot] = first + __ffs((int)sel) - 1;
}

// Ordered compaction of a cached row: thread t owns the `per` positions from
// t * per on (a multiple of four, at most 32) and marks those above and equal
// to tau in two bit masks; one scan over the workgroup of both counts gives it
// the slot of its first selected position, and the set bits go out in order.
// A thread reads its groups of four in an order that begins at a place of its
// own (whole rows of 128 bytes apart, all threads would meet in one bank).
// (Ballots over 256-position steps of a wave took 21 thousand cycles of the 47
// thousand of a 32768-position row, this 9.)  Places past the row hold key 0:
// above no tau, and equal to it only behind all the row's own keys that are,
// of which there are enough.  A slot is written only inside the row's k
// outputs.
template <int MOST>                              // groups of a thread
__device__ __forceinline__ void compact_cached(const uint32_t *keys, int n, int k, uint32_t tau, int need, int32_t *ws,
                                               int32_t *out)
{
    const int groups = (n + 4 * SEL_NT - 1) / (4 * SEL_NT), per = 4 * groups;
    const int first = (int)threadIdx.x * per, turn = (int)threadIdx.x % groups;
    uint32_t gt = 0, eq = 0;
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        if (i >= groups) break;                   // uniform
        int g = i + turn;
        g = g >= groups ? g - groups : g;
        const u32x4 q = *reinterpret_cast<const u32x4 *>(keys + first + 4 * g);
        uint32_t gt4 = 0, eq4 = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            gt4 |= q[c] > tau ? 1u << c : 0u;
            eq4 |= q[c] == tau ? 1u << c : 0u;
        }
        gt |= gt4 << (4 * g);
        eq |= eq4 << (4 * g);
    }
    int gt_b = 0, eq_b = 0;
    place_masks(gt, eq, first, k, need, gt_b, eq_b, ws, out);
}

// ---- a row too long for LDS: every pass re-reads the scores -----------------
__device__ __forceinline__ void select_uncached(const float *__restrict__ row, int n, int tail0, int k, int32_t *hist,
                                                int32_t *ws, int32_t *sel_s, int32_t *__restrict__ out)
{
    const int tid = threadIdx.x;
    auto key_of = [&](float f, int i) { return i >= n ? 0u : i >= tail0 ? TAIL_KEY : score_key(f); };
    // the scores of positions i .. i + 3 (i a multiple of four): one load inside the row, none past its end
    auto scores4 = [&](int i) {
        if (i + 4 <= n) return *reinterpret_cast<const f32x4 *>(row + i);
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (i + c < n) v[c] = row[i + c];
        return v;
    };
    uint32_t prefix = 0;
    int need = k;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const int nb = pass == 2 ? 1024 : 2048;
        const uint32_t hi = pass == 0 ? 0u : 0xffffffffu << (shift + (pass == 2 ? 10 : 11));
        for (int b0 = 4 * tid; b0 < n; b0 += 4 * SEL_GROUPS * SEL_NT) {
            f32x4 v[SEL_GROUPS];
#pragma unroll
            for (int j = 0; j < SEL_GROUPS; ++j) v[j] = scores4(b0 + 4 * j * SEL_NT);
#pragma unroll
            for (int j = 0; j < SEL_GROUPS; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int i = b0 + 4 * j * SEL_NT + c;
                    const uint32_t q = key_of(v[j][c], i);
                    if (i < n && (q & hi) == prefix) atomicAdd(&hist[(q >> shift) & (nb - 1)], 1);
                }
        }
        __syncthreads();
        int above;
        prefix |= (uint32_t)pick_bin(hist, nb, need, ws, sel_s, &above) << shift;
        need -= above;
    }
    // SEL_CAP positions at a time, 32 neighbours a thread (see compact_cached)
    const uint32_t tau = prefix;
    int gt_b = 0, eq_b = 0;
    for (int c0 = 0; c0 < n; c0 += SEL_CAP) {
        const int first = c0 + 32 * tid;
        uint32_t gt = 0, eq = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f32x4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = scores4(first + 16 * h + 4 * j);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int x = 16 * h + 4 * j + c;
                    const uint32_t q = key_of(v[j][c], first + x);    // 0 past the row
                    gt |= q > tau ? 1u << x : 0u;
                    eq |= q == tau ? 1u << x : 0u;
                }
        }
        place_masks(gt, eq, first, k, need, gt_b, eq_b, ws, out);
        __syncthreads();                          // ws is free again
    }
}

// Workgroup b takes rows b, b + G, b + 2G, ...: as many workgroups as run at
// once, so that clearing the histogram is paid once each.  CAP: the longest
// row kept in LDS.
template <int CAP>
__global__ __launch_bounds__(SEL_NT, CAP == SEL_CAP ? 4 : 8) void index_topk_kernel(const float *__restrict__ scores, int rows, int L,
                                                            long ld, const int32_t *__restrict__ lens,
                                                            int rows_per_len, int k, int tail,
                                                            int32_t *__restrict__ idx)
{
    constexpr int PER = CAP / (4 * SEL_NT);       // groups of four positions of a thread
    __shared__ __attribute__((aligned(16))) uint32_t keys[CAP];
    __shared__ int32_t hist[2048];
    __shared__ int32_t ws[SEL_WAVES];
    __shared__ int32_t sel_s[2];
    const int tid = threadIdx.x;
    for (int b = tid; b < 2048; b += SEL_NT) hist[b] = 0;
    int ahead = lens ? lens[rows_per_len == 1 ? blockIdx.x : blockIdx.x / rows_per_len] : L;
    for (uint32_t r = blockIdx.x; r < (uint32_t)rows; r += gridDim.x) {     // (unsigned: r passes 2^31 by less than a grid)
        const int n = min(max(ahead, 0), L);
        if (lens) {                               // the next row's length is on its way while this row is taken
            const uint32_t next = min(r + gridDim.x, (uint32_t)rows - 1u);
            ahead = lens[rows_per_len == 1 ? next : next / (uint32_t)rows_per_len];
        }
        int32_t *__restrict__ out = idx + (size_t)r * k;
        if (n <= k) {                             // the whole row, then -1
            // The first place is formed again for each row: kept over the row
            // loop it is spilled, and its reload waits for the last row's
            // stores (8192 rows of at most 64 positions: 15.1 us, 9.4 so).
            uint32_t j = tid;
            asm volatile("" : "+v"(j));
            for (; j < (uint32_t)k; j += SEL_NT) out[j] = (int)j < n ? (int)j : -1;
            continue;
        }
        const float *__restrict__ row = scores + (size_t)r * ld;
        const int tail0 = n - min(tail, k);       // positions >= tail0 are always kept
        __syncthreads();                          // the previous row is done with keys / hist
        if constexpr (CAP == SEL_CAP) {
            if (n > CAP) {                        // (it leaves the histogram clear, as it found it)
                select_uncached(row, n, tail0, k, hist, ws, sel_s, out);
                continue;
            }
        }
        {
            f32x4 v[PER];
            load_row(row, n, v);
            store_keys(row, n, tail0, v, keys, hist);
        }
        lds_barrier();
        // radix select: digits of 11, 11 and 10 bits, most significant first
        uint32_t prefix = 0;
        int need = k, above;
        prefix = (uint32_t)pick_bin(hist, 2048, need, ws, sel_s, &above) << 21;
        need -= above;
#pragma unroll 1
        for (int pass = 1; pass < 3; ++pass) {
            const int shift = pass == 1 ? 10 : 0;
            const int nb = pass == 2 ? 1024 : 2048;
            const uint32_t hi = 0xffffffffu << (shift + (pass == 2 ? 10 : 11));
            // groups of four positions, half the thread's groups loaded at a time
            constexpr int HALF = PER / 2;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 g[HALF];
#pragma unroll
                for (int j = 0; j < HALF; ++j)
                    g[j] = *reinterpret_cast<const u32x4 *>(keys + 4 * ((h * HALF + j) * SEL_NT + tid));
#pragma unroll
                for (int j = 0; j < HALF; ++j) {
                    const int i = 4 * ((h * HALF + j) * SEL_NT + tid);
                    if (4 * (h * HALF + j) * SEL_NT >= n) break;       // uniform: short rows have fewer groups
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (i + c < n && (g[j][c] & hi) == prefix) atomicAdd(&hist[(g[j][c] >> shift) & (nb - 1)], 1);
                }
            }
            lds_barrier();
            prefix |= (uint32_t)pick_bin(hist, nb, need, ws, sel_s, &above) << shift;
            need -= above;
        }
        compact_cached<PER>(keys, n, k, prefix, need, ws, out);
    }
}

hipError_t launch_index_topk(const float *scores, int rows, int L, long ld, const int32_t *lens, int rows_per_len,
                             int k, int tail, int32_t *idx, hipStream_t st)
{
    if (rows == 0) return hipSuccess;
    // two workgroups a CU where rows are short (2048 rows of 8192 scores: 46 us,
    // 59 with one; of 300 scores 32 and 44), with room for long ones else
    if (L <= SEL_SHORT)
        index_topk_kernel<SEL_SHORT><<<min(rows, 512), SEL_NT, 0, st>>>(scores, rows, L, ld, lens, rows_per_len, k, tail, idx);
    else
        index_topk_kernel<SEL_CAP><<<min(rows, 256), SEL_NT, 0, st>>>(scores, rows, L, ld, lens, rows_per_len, k, tail, idx);
    return hipGetLastError();
}

}  // namespace coli
