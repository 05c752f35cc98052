// attend.h -- attention of one new token per sequence over a paged
// key-value cache ("Add GLM-5.3-Flash (glm5next) support with ROCmFP mix
// qtypes (105/106)", section "MLA/DSA": softmax attention over the cached,
// or the selected, positions).
//
// Per query head q of sequence b, with t_p = scale q.k_p:
//   out = sum_p e^(t_p - m) v_p / sum_p e^(t_p - m),   m = max_p t_p
// in one pass over the cache: a wave keeps a running reference m of its
// query heads, the sum l and the unnormalised output O, and moves all three
// to a new reference when the maximum has grown (factor e^(m_old - m_new)).
// Parts of a sequence are joined by the same rule.  Exponents are taken to
// base 2 (t and m in units of log2 e).
//
// What bounds it: every key and value is read once and used by the few query
// heads of its cache head, so the cache's bytes at HBM rate.  Hence:
//  - no LDS staging: a wave takes 32 positions at a time, keys and values go
//    from global memory straight into the registers that feed the matrix
//    instructions, and a position's next read is issued as soon as its
//    registers are free (keys after the score products, values after the
//    output products), so every wave always has 32 rows in flight;
//  - the work (32-position steps of all sequences and heads in one line) is
//    cut into equal ranges, one a workgroup, whatever the sequences' lengths
//    (read on the device); a row cut by a range's border leaves a part in the
//    workspace, and a second kernel joins the parts.
// Measured, bf16, 8 cache heads of width 128 (a device copy moves 4.9 TB/s):
// one sequence of 131071 positions 97 us and 6 for the join (537 MB, 5.5 TB/s
// in the kernel), 64 of 0 to 32768 positions 165 + 8 us (882 MB, 5.3 TB/s),
// one of 777 positions 7.5 + 4 us (latencies).
#pragma once

#include "device_common.h"
#include "kernels.h"

namespace coli {

constexpr int KV_NT = 256;                    // threads per workgroup (4 waves)
constexpr int KV_WAVES = KV_NT / 64;
constexpr int KV_STEP = 32;                   // positions per step of a wave
constexpr int KV_QT = 16;                     // query heads per matrix tile
constexpr int KV_MAX_WG = 512;                // most ranges

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short bf16x8s __attribute__((ext_vector_type(8)));

// What a launch takes of the sequences: all positions; those behind the pages
// that a sequence shares; or those pages, a group of sequences in the place of
// a sequence and all its members' query heads in the place of one's.
enum KvPart { KV_ALL, KV_OWN, KV_PREFIX };

// Sequences of group g: the groups are a partition of the batch.
// (Loads without branches, so that they are in flight together.)
__device__ __forceinline__ int kv_group_first(const AttnLaunch &a, int g)
{
    const int at = a.group_start[g];
    return g == 0 ? 0 : min(max(at, 0), a.B);
}
__device__ __forceinline__ int kv_group_end(const AttnLaunch &a, int g)
{
    const int at = a.group_start[g + 1];
    return g + 1 == a.n_groups ? a.B : min(max(at, 0), a.B);
}
// Pages that sequence b shares with its group, and the ones that its own part
// leaves to it: none where the sequence ends before them (it is then taken
// whole as its own, and what the group finds for it does not count).
__device__ __forceinline__ int kv_shared(const AttnLaunch &a, int b) { return min(max(a.shared[b], 0), a.max_pages); }
__device__ __forceinline__ int kv_left(const AttnLaunch &a, int b)
{
    const int pages = kv_shared(a, b);
    return min(max(a.lens[b], 0), a.cap) >= pages << a.page_shift ? pages : 0;
}

// Entries of sequence (or group) b: positions, or listed ones.
template <KvPart PART = KV_ALL>
__device__ __forceinline__ int kv_len(const AttnLaunch &a, int b)
{
    if constexpr (PART == KV_OWN) return min(max(a.lens[b], 0), a.cap) - (kv_left(a, b) << a.page_shift);
    if constexpr (PART == KV_PREFIX) {
        const int first = kv_group_first(a, b), end = kv_group_end(a, b);
        const int pages = kv_shared(a, min(first, a.B - 1));
        return first < end ? pages << a.page_shift : 0;
    }
    return a.idx ? a.idx_k : min(max(a.lens[b], 0), a.cap);
}

// Sequences (or groups), and their rows: query tiles of all cache heads.
template <KvPart PART>
__device__ __forceinline__ int kv_items(const AttnLaunch &a) { return PART == KV_PREFIX ? a.n_groups : a.B; }
template <KvPart PART>
__device__ __forceinline__ int kv_tiles(const AttnLaunch &a, int b)
{
    if constexpr (PART != KV_PREFIX) return a.q_tiles;
    const int queries = (kv_group_end(a, b) - kv_group_first(a, b)) * (a.Hq / a.Hkv);
    return (queries + a.tile_rows - 1) / a.tile_rows;
}
__device__ __forceinline__ int kv_steps(int n) { return (n + KV_STEP - 1) / KV_STEP; }

// Work is counted in units: the steps of a row (a cache head's query tile of
// one sequence), rounded up to whole KV_ROW_UNITS.  A short row costs its
// latencies and not its steps (a range of eight one-step rows took 40 us),
// and a border just before a row's end would give one workgroup two rows'
// latencies (25 against 16 thousand cycles).  128 sequences of 1 to 8192
// positions, 8 cache heads of 128: 140 us, in units of single steps 193.
constexpr int KV_ROW_UNITS = 8;
__device__ __forceinline__ int kv_units(int n) { return (kv_steps(n) + KV_ROW_UNITS - 1) / KV_ROW_UNITS * KV_ROW_UNITS; }

// Units of all sequences before b, and of all (per row of a sequence).  Every
// wave computes it by itself: no barriers, and one load for up to 64
// sequences.  Of groups: the units of all their rows.
template <KvPart PART = KV_ALL>
__device__ __forceinline__ int kv_item_units(const AttnLaunch &a, int b)
{
    const int units = kv_units(kv_len<PART>(a, b));
    return PART == KV_PREFIX ? units * a.Hkv * kv_tiles<PART>(a, b) : units;
}
template <KvPart PART = KV_ALL>
__device__ __forceinline__ void kv_prefix(const AttnLaunch &a, int b, int *before, int *total)
{
    if (PART == KV_ALL && a.idx) {
        const int per = kv_units(a.idx_k);
        *before = b * per;
        *total = a.B * per;
        return;
    }
    const int lane = threadIdx.x & 63;
    int lo = 0, all = 0;
    bool falls = false;
    for (int i = lane; i < kv_items<PART>(a); i += 64) {
        const int st = kv_item_units<PART>(a, i);
        all += st;
        lo += (i < b) ? st : 0;
        if constexpr (PART == KV_PREFIX) falls |= kv_group_end(a, i) < kv_group_first(a, i);
    }
    // Borders that fall somewhere can count sequences any number of times, past 2^31 units: nothing is taken.
    if (PART == KV_PREFIX && __ballot(falls)) lo = all = 0;
    *before = __builtin_amdgcn_readlane(wave_scan_incl(lo), 63);
    *total = __builtin_amdgcn_readlane(wave_scan_incl(all), 63);
}

// Units of one workgroup's range: half of KV_ROW_UNITS, or whole ones, so that
// borders and rows' ends meet where the work is small.
__device__ __forceinline__ int kv_range(const AttnLaunch &a, int units)
{
    const int even = (units + a.n_wg - 1) / a.n_wg;
    return even <= a.min_units ? a.min_units : (even + KV_ROW_UNITS - 1) / KV_ROW_UNITS * KV_ROW_UNITS;
}

// A workgroup's range: units u .. u_end - 1, beginning with unit s0 (a step,
// or past the last one) of row `row` of sequence b.
struct KvRange {
    int u, u_end, b, n, steps, row, s0;
};

// False: the range is empty.  R rows a sequence (groups: 1, their units are
// all rows').  The same for every wave.
template <KvPart PART = KV_ALL>
__device__ __forceinline__ bool kv_first(const AttnLaunch &a, int R, KvRange &rg, int blk = blockIdx.x)
{
    if constexpr (PART != KV_ALL) {           // up to 64 items: in one look at them
        if (kv_items<PART>(a) <= 64) {
            const int lane = threadIdx.x & 63, i = min(lane, kv_items<PART>(a) - 1);
            const bool some = lane < kv_items<PART>(a);
            const int n = some ? kv_len<PART>(a, i) : 0;
            const int st = kv_units(n) * (PART == KV_PREFIX ? a.Hkv * kv_tiles<PART>(a, i) : 1);
            if (PART == KV_PREFIX && __ballot(kv_group_end(a, i) < kv_group_first(a, i))) return false;
            const int incl = wave_scan_incl(st), total = __builtin_amdgcn_readlane(incl, 63) * R;
            const int range = kv_range(a, total), u = blk * range;
            if (u >= total) return false;
            const int x = __ffsll((unsigned long long)__ballot(u < incl * R)) - 1;
            const int at = u - __builtin_amdgcn_readlane(incl - st, x) * R;
            rg.u = u;
            rg.u_end = min(u + range, total);
            rg.b = x;
            rg.n = __builtin_amdgcn_readlane(n, x);
            rg.steps = kv_steps(rg.n);
            rg.row = at / kv_units(rg.n);
            rg.s0 = at - rg.row * kv_units(rg.n);
            return true;
        }
    }
    int before, total;
    kv_prefix<PART>(a, 0, &before, &total);
    total *= R;
    const int range = kv_range(a, total);
    const int u = blk * range;         // below total + n_wg * (KV_ROW_UNITS + 1), and 2^31 by the host's check
    if (u >= total) return false;
    int base = 0;
    if (PART == KV_ALL && a.idx) {
        const int per = kv_units(a.idx_k) * R;
        rg.b = u / per;
        base = rg.b * per;
    } else {
        const int lane = threadIdx.x & 63;
        int sum = 0;                          // units (per row) before this chunk of sequences
        for (int c = 0;; c += 64) {
            const int st = (c + lane < kv_items<PART>(a)) ? kv_item_units<PART>(a, c + lane) : 0;
            const int incl = wave_scan_incl(st) + sum;
            const uint64_t here = __ballot(u < incl * R);
            if (here) {                       // the first lane that ends behind u (u < total: there is one)
                const int x = __ffsll((unsigned long long)here) - 1;
                rg.b = c + x;
                base = __builtin_amdgcn_readlane(incl - st, x) * R;
                break;
            }
            sum = __builtin_amdgcn_readlane(incl, 63);
        }
    }
    rg.u = u;
    rg.u_end = min(u + range, total);
    rg.n = kv_len<PART>(a, rg.b);
    rg.steps = kv_steps(rg.n);
    const int per = kv_units(rg.n);
    rg.row = (u - base) / per;
    rg.s0 = (u - base) - rg.row * per;
    return true;
}

// A workgroup's range, or (direct) its row, which may be empty.
template <KvPart PART = KV_ALL>
__device__ __forceinline__ bool kv_begin(const AttnLaunch &a, int R, KvRange &rg, int blk = blockIdx.x)
{
    if (!a.direct) return kv_first<PART>(a, PART == KV_PREFIX ? 1 : R, rg, blk);
    rg.b = blk / R;
    rg.row = blk - rg.b * R;
    rg.n = kv_len<PART>(a, rg.b);
    rg.steps = kv_steps(rg.n);
    rg.u = rg.s0 = 0;
    rg.u_end = max(rg.steps, 1);
    return true;
}

// The next row of a range (past the last sequence: one that is never taken).
template <KvPart PART = KV_ALL>
__device__ __forceinline__ void kv_next_row(const AttnLaunch &a, int R, int &b, int &n, int &steps, int &row)
{
    if (++row < (PART == KV_PREFIX ? a.Hkv * kv_tiles<PART>(a, b) : R)) return;
    row = 0;
    do {
        ++b;
        n = b < kv_items<PART>(a) ? kv_len<PART>(a, b) : 1;
    } while (n == 0);
    steps = kv_steps(n);
}

// A group's row, a query tile: cache head, the first of its queries and how
// many the cache head has in all.  Query i of a cache head is row kv_query_row
// of q.
struct KvTileOf {
    int h, q0, queries;
};
__device__ __forceinline__ KvTileOf kv_tile_of(const AttnLaunch &a, int g, int row)
{
    const int tiles = kv_tiles<KV_PREFIX>(a, g);
    KvTileOf t;
    t.h = tiles == 1 ? row : row / tiles;
    t.q0 = (row - t.h * tiles) * a.tile_rows;
    t.queries = (kv_group_end(a, g) - kv_group_first(a, g)) * (a.Hq / a.Hkv);
    return t;
}
__device__ __forceinline__ size_t kv_query_row(const AttnLaunch &a, int first, int h, int i)
{
    const int G = a.Hq / a.Hkv, x = i / G;
    return (size_t)(first + x) * a.Hq + h * G + (i - x * G);
}

__device__ __forceinline__ int kv_pool_row(const AttnLaunch &a, int pg, int h, int p)
{
    return (int)((((uint32_t)pg * (uint32_t)a.Hkv + (uint32_t)h) << a.page_shift) +
                 (uint32_t)(p & ((1 << a.page_shift) - 1)));
}

// Pool row of entry e < end of sequence b's positions (of its list, where
// there is one) for cache head h; -1: hidden.  No branches, and the table is
// read before the length is known: its loads wait for nothing.
template <KvPart PART = KV_ALL>
__device__ __forceinline__ int kv_row(const AttnLaunch &a, int b, int h, int end, int len, int e)
{
    int p = e;
    if (PART == KV_ALL && a.idx) p = a.idx[(size_t)b * a.idx_k + min(e, a.idx_k - 1)];
    int at = min(max(p, 0), a.cap - 1);
    size_t entry;
    if constexpr (PART == KV_ALL) {
        entry = (size_t)b * a.max_pages + (at >> a.page_shift);
    } else {
        const int first = PART == KV_OWN ? kv_left(a, b) : 0;              // (of a row with entries: a page is left)
        at = min(at, max(a.cap - (first << a.page_shift), 1) - 1);
        entry = (size_t)(PART == KV_PREFIX ? kv_group_first(a, b) : b) * a.max_pages + first + (at >> a.page_shift);
    }
    const int pg = a.table[entry];
    const bool ok = e < end && p >= 0 && p < len && pg >= 0 && pg < a.n_pages;
    return ok ? kv_pool_row(a, pg, h, at) : -1;
}

// ---- operands -----------------------------------------------------------------
// A lane reads 16 bytes of a row at a time: EPL elements.  Keys: lane (j, g)
// (j = lane & 15, g = lane >> 4) holds elements (4 c + g) EPL .. of key j,
// chunk c; the query is read the same way, so whatever slots the matrix
// instruction gives to a lane's elements, both operands agree.  Values: lane
// (j, g) holds elements (16 h + j) VE .. of the 8 positions 4 g + 0..3 and
// 16 + 4 g + 0..3, which are the positions whose weights the score product
// left in the lanes of the same g.
template <bool BF16>
struct KvType;
template <>
struct KvType<true> {
    using T = uint16_t;
    static constexpr int EPL = 8;
};
template <>
struct KvType<false> {
    using T = float;
    static constexpr int EPL = 4;
};

// What a key's columns past its width read, and hidden positions of the latent
// kernel: zeros, since a zero of the query would not stop an infinity there.
static __device__ const u32x4 kv_zeros[72] = {};

// A score in units of log2 e.  The factor's small part meets finite numbers
// only: it may be of the other sign, and an infinite score keeps its own.
__device__ __forceinline__ float kv_scaled(const AttnLaunch &a, float score)
{
    return fmaf(score, a.scale_hi, __builtin_amdgcn_fmed3f(score, -a.scale_cap, a.scale_cap) * a.scale_lo);
}

__device__ __forceinline__ bf16x8 as_bf16(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    return (uint32_t)f32_to_bf16_bits(lo) | ((uint32_t)f32_to_bf16_bits(hi) << 16);
}

template <bool BF16, int DK, int DV>
struct KvTile {
    using KT = KvType<BF16>;
    using T = typename KT::T;
    static constexpr int EPL = KT::EPL;
    static constexpr int KC = DK / (4 * EPL);                      // key chunks of a lane
    static constexpr int VE = (DV >= 16 * EPL) ? EPL : DV / 16;    // value elements a lane reads at once
    static constexpr int VC = DV / (16 * VE);                      // value chunks of a lane
    static constexpr int VW = VE * (int)sizeof(T) / 4;             // dwords of a value chunk
    static_assert(VW == 4 || VW == 2, "8 or 16 bytes of a value row");
};

// lse of a query row, and its reference and 1 / sum for the running weights.
// A sum is 0 for an empty row only, and a NaN for one that met a NaN.
__device__ __forceinline__ float kv_inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ void kv_write_lse(const AttnLaunch &a, size_t q, float m, float l)
{
    if (a.lse) a.lse[q] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}
__device__ __forceinline__ void kv_write_stats(const AttnLaunch &a, size_t q, float m, float l)
{
    kv_write_lse(a, q, m, l);
    if (a.stats) {
        a.stats[2 * q] = m == -INFINITY ? 0.f : m;
        a.stats[2 * q + 1] = kv_inverse(l);
    }
}

// (max, +) over the four lanes of a query head (lanes j, j + 16, j + 32, j + 48).
__device__ __forceinline__ float quad_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float quad_sum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Zeros for the rows of an empty sequence, by the whole workgroup.
__device__ __forceinline__ void kv_write_empty(const AttnLaunch &a, size_t qrow, int nq)
{
    for (size_t i = threadIdx.x; i < (size_t)nq * a.Dv; i += blockDim.x) {
        if (a.bf16) ((uint16_t *)a.out)[qrow * a.Dv + i] = 0;
        else ((float *)a.out)[qrow * a.Dv + i] = 0.f;
    }
    if ((int)threadIdx.x < nq) kv_write_stats(a, qrow + threadIdx.x, -INFINITY, 0.f);
}

// NW waves; `a.direct`: a workgroup per row, none of them cut.
// PART other than KV_ALL: rows that are not cut are left as parts too, by their
// queries (a.full_o, a.full_ml).
template <bool BF16, int DK, int DV, int NW, KvPart PART>
__device__ __forceinline__ void attn_rows(const AttnLaunch &a, int blk)
{
    using KT = KvTile<BF16, DK, DV>;
    using T = typename KT::T;
    constexpr int EPL = KT::EPL, KC = KT::KC, VE = KT::VE, VC = KT::VC, VW = KT::VW;
    // BIG: too wide for a step's rows in registers; keys are taken KP chunks at
    // a time, values chunk by chunk, each read one ahead of its products (fp32,
    // 32 sequences of 4096 positions, 8 heads of 256: 662 us with the whole
    // rows, which spill 57 registers, 354 so).
    constexpr bool BIG = DK > (BF16 ? 256 : 192);
    // KP: 32 sequences of 4096 positions at width 256, 16 latent ones of 4096
    // at 576 and 320 elements (64 heads): 354, 140, 80 us with four chunks, 144
    // with six at 576, 80 with five at 320.
    constexpr int KP = BIG ? 4 : KC;
    static_assert(!BIG || (KC % KP == 0 && !BF16), "whole groups; bf16 takes the LDS kernel");
    constexpr int RS = DV + 4;                // padded row of the join buffer
    __shared__ __attribute__((aligned(16))) float red[NW][KV_QT][RS];
    __shared__ float red_m[NW][KV_QT], red_l[NW][KV_QT];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int j = lane & 15, g = lane >> 4;
    const int G = a.Hq / a.Hkv;
    const int R = a.Hkv * a.q_tiles;

    KvRange rg;
    if (!kv_begin<PART>(a, R, rg, blk)) return;
    int u = rg.u, b = rg.b, n = rg.n, steps = rg.steps, row = rg.row, s0 = rg.s0;
    const int u_begin = u, u_end = rg.u_end;

    const T *kpool = (const T *)a.k;
    const T *vpool = (const T *)(a.v ? a.v : a.k);
    const int vstride = a.v ? a.Dv : a.Dk;
    const int key_chunks = (a.Dk + 4 * EPL - 1) / (4 * EPL), full_chunks = a.Dk / (4 * EPL);

    for (; u < u_end; u += kv_units(n) - s0, s0 = 0, kv_next_row<PART>(a, R, b, n, steps, row)) {
        const int s1 = min(steps, s0 + (u_end - u));
        int h, q0, nq;                        // (nq: query heads of this tile)
        if constexpr (PART == KV_PREFIX) {
            const KvTileOf t = kv_tile_of(a, b, row);
            h = t.h, q0 = t.q0, nq = min(KV_QT, t.queries - q0);
        } else {
            h = a.q_tiles == 1 ? row : row / a.q_tiles, q0 = (row - h * a.q_tiles) * KV_QT;
            nq = min(KV_QT, G - q0);
        }
        const size_t qrow = (size_t)b * a.Hq + h * G + q0;
        if (s0 >= steps) {                    // a row's units past its steps, or (direct) an empty row
            if (a.direct) {
                if (PART == KV_ALL) kv_write_empty(a, qrow, nq);
                return;
            }
            continue;
        }
        const int len = PART == KV_ALL ? min(max(a.lens[b], 0), a.cap) : n;
        size_t query = qrow + j;              // the lane's
        if constexpr (PART == KV_PREFIX) query = kv_query_row(a, kv_group_first(a, b), h, q0 + min(j, nq - 1));

        // the query tile: lane (j, g) holds query j's elements as a key's
        u32x4 qf[KC];
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const int d = (4 * c + g) * EPL;
            qf[c] = u32x4{0, 0, 0, 0};
            if (j < nq && d < a.Dk)
                qf[c] = *reinterpret_cast<const u32x4 *>((const T *)a.q + query * a.Dk + d);
        }
        f32x4 o[VC][VE];
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int e = 0; e < VE; ++e) o[c][e] = f32x4{0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, l = 0.f;

        // pool row of position `lane & 31` of step s (-1: hidden)
        const int end = min(n, s1 * KV_STEP);
        auto rows_of = [&](int s) { return kv_row<PART>(a, b, h, end, len, s * KV_STEP + (lane & 31)); };
        u32x4 kf[2][BIG ? 2 * KP : KC];
        auto load_keys = [&](int rows, int c0 = 0) {      // (BIG: KP chunks from c0 on, into their half of the buffer)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int r = max(__shfl(rows, 16 * t + j), 0);
                const T *p = kpool + (size_t)r * a.Dk + g * EPL;
                // All chunks inside the row (fp32 width 128, 32 sequences of 4096 positions, 8 heads: 40.8 us, 43.0 the other
                // way; in the widest kernel a second way sends the buffer to scratch, 440 us against 143).
                if (DK <= 256 && c0 + KP <= full_chunks) {
#pragma unroll
                    for (int x = 0; x < KP; ++x)
                        kf[t][BIG ? (c0 + x) % (2 * KP) : c0 + x] = *reinterpret_cast<const u32x4 *>(p + 4 * (c0 + x) * EPL);
                    continue;
                }
#pragma unroll
                for (int x = 0; x < KP; ++x) {
                    const int c = c0 + x;                 // past the row's width: zeros
                    if (BIG || c < key_chunks)            // (the address space is named: with flat loads 300 -> 400 us at width 192)
                        kf[t][BIG ? c % (2 * KP) : c] = *(const __attribute__((address_space(1))) u32x4 *)(
                            (4 * c + g) * EPL < a.Dk ? (uint64_t)(p + 4 * c * EPL) : (uint64_t)kv_zeros);
                }
            }
        };
        uint32_t vf[BIG ? 2 : VC][8][VW];
        auto load_values = [&](int rows, int c0 = 0) {    // (BIG: chunk c0)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = max(__shfl(rows, 16 * (i >> 2) + 4 * g + (i & 3)), 0);
                const T *p = vpool + (size_t)r * vstride;
#pragma unroll
                for (int x = 0; x < (BIG ? 1 : VC); ++x) {
                    const int c = BIG ? c0 : x, to = BIG ? c0 & 1 : x;
                    const int d = (16 * c + j) * VE;      // past the value's width: columns that are not written
                    const T *src = p + (d < a.Dv ? d : 0);
                    if constexpr (VW == 4) {
                        const u32x4 v = *reinterpret_cast<const u32x4 *>(src);
#pragma unroll
                        for (int w = 0; w < 4; ++w) vf[to][i][w] = v[w];
                    } else {
                        const u32x2 v = *reinterpret_cast<const u32x2 *>(src);
                        vf[to][i][0] = v[0];
                        vf[to][i][1] = v[1];
                    }
                }
            }
        };
        // what stands in hidden rows (NaN, infinities) must not count
        auto clear_hidden = [&](int rows, int first, int last) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (__shfl(rows, 16 * (i >> 2) + 4 * g + (i & 3)) < 0) {
#pragma unroll
                    for (int c = first; c < last; ++c)
#pragma unroll
                        for (int x = 0; x < VW; ++x) vf[c][i][x] = 0u;
                }
        };

        int s = s0 + wave;
        int rows = rows_of(s), rows_next = rows_of(s + NW);
        if (!BIG && s < s1) {
            load_keys(rows);
            load_values(rows);
        }
        for (; s < s1; s += NW) {
            const bool more = s + NW < s1;
            // ---- scores: D[key][query] = K Q^T, two tiles of 16 keys ----
            // fp32 parts of wide rows: two sums, which halves what a long chain rounds away (rows of 512: outputs 8.3e-7
            // off, 2.0e-6 with one; the times are the same, but 64-wide rows would lose a wave a SIMD: 18.6 -> 21.4 us).
            constexpr int SUMS = !BF16 && PART != KV_ALL && DK > 64 ? 2 : 1;
            f32x4 sc[2], sc2[2];
            sc[0] = sc[1] = sc2[0] = sc2[1] = f32x4{0.f, 0.f, 0.f, 0.f};
            auto product = [&](const u32x4 &k0, const u32x4 &k1, int c) {
                if constexpr (BF16) {
                    sc[0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(k0), as_bf16(qf[c]), sc[0], 0, 0, 0);
                    sc[1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(k1), as_bf16(qf[c]), sc[1], 0, 0, 0);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        f32x4 *d = SUMS == 2 && e & 1 ? sc2 : sc;
                        d[0] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k0[e]), __uint_as_float(qf[c][e]), d[0], 0, 0, 0);
                        d[1] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k1[e]), __uint_as_float(qf[c][e]), d[1], 0, 0, 0);
                    }
                }
            };
            if constexpr (BIG) {
                load_keys(rows, 0);
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    if (c % KP == 0 && c + KP < KC) load_keys(rows, c + KP);
                    product(kf[0][c % (2 * KP)], kf[1][c % (2 * KP)], c);
                    if (c % KP == KP - 1) __builtin_amdgcn_sched_barrier(0);
                }
            } else {
#pragma unroll
                for (int c = 0; c < KC; ++c)
                    if (c < key_chunks) product(kf[0][c], kf[1][c], c);
            }
            if constexpr (SUMS == 2) {
                sc[0] += sc2[0];
                sc[1] += sc2[1];
            }
            const int rows_now = rows;
            rows = rows_next;
            if (!BIG && more) load_keys(rows);
            if constexpr (BIG) load_values(rows_now);
            rows_next = rows_of(s + 2 * NW);

            // ---- weights: lane (j, g) holds query j, positions 16 t + 4 g + r ----
            float t2[8];
            const uint64_t hidden = __ballot(rows_now < 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) t2[i] = kv_scaled(a, sc[i >> 2][i & 3]);
            if (hidden) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (__shfl(rows_now, 16 * (i >> 2) + 4 * g + (i & 3)) < 0) t2[i] = -INFINITY;
            }
            if (PART == KV_ALL && a.scores) {
                // raw scores for the running weights (query j's row)
                if (j < nq) {
                    float *dst = a.scores + (qrow + j) * a.s_ld + s * KV_STEP + 4 * g;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        *reinterpret_cast<f32x4 *>(dst + 16 * t) = f32x4{t2[4 * t], t2[4 * t + 1], t2[4 * t + 2], t2[4 * t + 3]};
                }
            }
            float mx = t2[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) mx = fmaxf(mx, t2[i]);
            // The reference moves only when a score passes it by 2^8: weights
            // stay below 256 and the sums far inside fp32.
            if (__ballot(mx > m + 8.f)) {
                const float mn = fmaxf(m, quad_max(mx));
                const float f = (mn == -INFINITY) ? 1.f : __builtin_amdgcn_exp2f(m - mn);
                m = mn;
                l *= f;
#pragma unroll
                for (int c = 0; c < VC; ++c)
#pragma unroll
                    for (int e = 0; e < VE; ++e) o[c][e] *= f;
            }
            const float ref = (m == -INFINITY) ? 0.f : m;
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[i] = __builtin_amdgcn_exp2f(t2[i] - ref);
                l += w[i];
            }
            // ---- output: O^T[value column][query] += V^T w ----
            if (!BIG && hidden) clear_hidden(rows_now, 0, BIG ? 0 : VC);
            if constexpr (BF16) {
                // each weight as two bf16 parts: 16 bits of it enter the products
                u32x4 hi, lo;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    hi[x] = pack_bf16(w[2 * x], w[2 * x + 1]);
                    lo[x] = pack_bf16(w[2 * x] - __uint_as_float(hi[x] << 16),
                                      w[2 * x + 1] - __uint_as_float(hi[x] & 0xffff0000u));
                }
#pragma unroll
                for (int c = 0; c < VC; ++c)
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        // column e of the lane's 8 x VE block: element e of each of the 8 rows
                        u32x4 col;
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            col[x] = __builtin_amdgcn_perm(vf[c][2 * x + 1][e >> 1], vf[c][2 * x][e >> 1],
                                                           (e & 1) ? 0x07060302u : 0x05040100u);
                        o[c][e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(col), as_bf16(hi), o[c][e], 0, 0, 0);
                        o[c][e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(col), as_bf16(lo), o[c][e], 0, 0, 0);
                    }
            } else {
#pragma unroll
                for (int c = 0; c < VC; ++c) {
                    if constexpr (BIG) {
                        if (c + 1 < VC) load_values(rows_now, c + 1);
                        if (hidden) clear_hidden(rows_now, c & 1, (c & 1) + 1);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int e = 0; e < VE; ++e)
                            o[c][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(vf[BIG ? c & 1 : c][i][e]), w[i],
                                                                          o[c][e], 0, 0, 0);
                    if constexpr (BIG) __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (!BIG && more) load_values(rows);
        }

        // ---- the waves' parts become one ----
        l = quad_sum(l);
        if (g == 0) {
            red_m[wave][j] = m;
            red_l[wave][j] = l;
        }
        if (j < nq) {
#pragma unroll
            for (int c = 0; c < VC; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int e = 0; e < VE; ++e) red[wave][j][(16 * c + 4 * g + r) * VE + e] = o[c][e][r];
        }
        __syncthreads();
        const bool whole = s0 == 0 && s1 == steps;
        const int slot = 2 * blk + (u == u_begin ? 0 : 1);
        // four columns of a query a thread
        for (int i = tid; i < nq * (DV / 4); i += 64 * NW) {
            const int q = i / (DV / 4), d = i % (DV / 4) * 4;
            if (d >= a.Dv) continue;
            float mq = red_m[0][q], lq = 0.f;
#pragma unroll
            for (int w = 1; w < NW; ++w) mq = fmaxf(mq, red_m[w][q]);
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = red_m[w][q] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(red_m[w][q] - mq);
                lq += red_l[w][q] * f;
                v += *reinterpret_cast<const f32x4 *>(&red[w][q][d]) * f;
            }
            if (PART != KV_ALL && whole) {
                const size_t at = PART == KV_PREFIX ? kv_query_row(a, kv_group_first(a, b), h, q0 + q) : qrow + q;
                *reinterpret_cast<f32x4 *>(a.full_o + at * a.Dv + d) = v;
                if (d == 0) {
                    a.full_ml[2 * at] = mq;
                    a.full_ml[2 * at + 1] = lq;
                }
            } else if (whole) {
                const float inv = kv_inverse(lq);
                const size_t at = (qrow + q) * a.Dv + d;
                if constexpr (BF16)
                    *reinterpret_cast<u32x2 *>((uint16_t *)a.out + at) =
                        u32x2{pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv)};
                else *reinterpret_cast<f32x4 *>((float *)a.out + at) = v * inv;
                if (d == 0) kv_write_stats(a, qrow + q, mq, lq);
            } else {
                *reinterpret_cast<f32x4 *>(a.part_o + ((size_t)slot * KV_QT + q) * a.Dv + d) = v;
                if (d == 0) {
                    a.part_ml[((size_t)slot * KV_QT + q) * 2] = mq;
                    a.part_ml[((size_t)slot * KV_QT + q) * 2 + 1] = lq;
                }
            }
        }
        if (a.direct) return;
        __syncthreads();                      // the join buffer is free again
    }
}

template <bool BF16, int DK, int DV, int NW>
__global__ __launch_bounds__(64 * NW) void attn_kernel(AttnLaunch a)
{
    attn_rows<BF16, DK, DV, NW, KV_ALL>(a, blockIdx.x);
}

// Where the parts of a sequence's row are: ranges w0 .. w1 hold some of it (w0 = w1: one
// holds all, and has written the row's results); the first part's slot, the
// later ranges' being their first ones.
struct KvParts {
    int steps, w0, w1, first;
    __device__ __forceinline__ int slot(int w) const { return w == w0 ? first : 2 * w; }
};
template <KvPart PART = KV_ALL>
__device__ __forceinline__ KvParts kv_parts(const AttnLaunch &a, int b, int row, int before, int total)
{
    const int R = a.Hkv * a.q_tiles, n = kv_len<PART>(a, b);
    KvParts p{kv_steps(n), 0, 0, 0};
    if (p.steps == 0) return p;
    const int range = kv_range(a, total * R);
    const int u0 = before * R + row * kv_units(n);
    p.w0 = u0 / range;
    p.w1 = (u0 + p.steps - 1) / range;
    p.first = 2 * p.w0 + (u0 == p.w0 * range ? 0 : 1);
    return p;
}

// ---- wide latent caches -------------------------------------------------------
// One latent row of up to 576 elements serves all query heads of its cache
// head (up to 128 a workgroup) as key and as value, so the products weigh as
// much as the reading: 64 heads are 100 products a byte.  Hence each row is
// brought into LDS once (copies that pass no registers, a ring of four
// 32-position stages) and every wave takes 32 query heads on 32 x 32 x 16
// matrix tiles (twice the rate of the 16 x 16 x 32 form):
//   scores  D[key][query] = K Q^T       36 tiles a stage, keys read as rows
//   output  O^T[column][query] += V^T w  32 tiles a stage and part of the
//           weights, values read column-wise out of the same rows (the LDS
//           transposing read: 16 lanes take a block of 4 rows x 16 columns
//           and each gets one column's 4 rows)
// A lane's 16 scores belong to one query, so the softmax needs one lane
// exchange, and the weights are in place as the second product's operand:
// its reduction slots are given to the positions in the order the lanes hold
// them.  O^T (256 registers) and the queries (144) stay in registers.
// Waves that share a stage: WQ = 4, 2, 1 query tiles for up to 128, 64, 32
// heads, fewer where the work is small (attn_plan); with WQ < 4 the waves also split the positions (WK = 4 / WQ stages
// at a time), and the parts are joined in LDS at the end of a row.
// LDS layout of a stage: the columns that are values too (DV of them) first,
// row after row, then the keys' last 64.  A row of the first part is whole
// bank rounds, so chunk c (16 bytes) of row r sits at c with its low four
// bits XORed by r's low bits (1, 0, 3, 2): 16 rows of one chunk (scores) and
// 4 rows of 4 chunks (output) both fall in distinct banks.  A copy
// instruction brings one row (or two of 256 columns), so its address is
// uniform: a few scalar instructions, which go between the products.
// Measured, 576 / 512 elements: 32 sequences of 8000 to 32768 positions, 128
// heads, 246-273 us (658 MB and 157 GFLOP of the formula, 231 with the weights'
// second parts).  Bound by the order of a stage's work: scores, weights and
// output follow one another, on one wave a SIMD, so the matrix cores are busy
// half of the time that the CUs are (and HBM is at half its rate).  64 heads
// over 64 rows of 2048 listed positions: 53 us (151 MB, 2.9 TB/s: a workgroup
// starts, takes 16 stages and leaves a part), and 9 for the join.
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int KW_ROWS = 32;                   // positions of a stage
constexpr int KW_MAX_WG = 256;                // ranges: one workgroup per CU, the ring fills its LDS
constexpr int KW_RING = 4;                    // stages in LDS
constexpr int KW_BLOCK = 32;                  // stages whose rows are looked up at a time

template <int N>
struct KwInt {
    static constexpr int value = N;
};

__device__ __forceinline__ int kw_swz(int row) { return ((row & 3) << 2) | ((row >> 2) & 3); }

template <int N>
__device__ __forceinline__ void kw_wait_copies()
{
    static_assert(N >= 0 && N <= 63, "vmcnt");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

__device__ __forceinline__ void kw_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// 16 bytes of each lane's address to LDS, lane after lane from byte `dst`
// (uniform): the address uniform with an offset for each lane, or the lane's
// own.  In assembler, and counted by hand (kw_wait_copies), because the
// compiler lets every transposing read wait for all copies in flight where it
// knows of them.  There is no register output, and the compiler has no use of
// its own for m0 here; the barriers order what is written.
__device__ __forceinline__ void kw_copy(uint64_t base, uint32_t off, uint32_t dst)
{
    // five wait states between the lane read that formed the base and its use as an address
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %0" ::"s"(base), "v"(off),
                 "s"(__builtin_amdgcn_readfirstlane(dst)));
}
__device__ __forceinline__ void kw_copy(uint64_t src, uint32_t dst)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src),
                 "s"(__builtin_amdgcn_readfirstlane(dst)));
}

// lane i's value (i uniform)
__device__ __forceinline__ uint64_t kw_lane(uint64_t v, int i)
{
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, i);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), i);
    return (uint64_t)hi << 32 | lo;
}

// d += a b on vector registers.  The compiler gives every product of a kernel
// its accumulator in the 256 accumulation registers; with the output's 256
// there, the scores must be in the others.  Two wait states: an operand may
// have been written by the instruction before.
__device__ __forceinline__ void kw_mfma_v(f32x16 &d, bf16x8 a, bf16x8 b)
{
    asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(d) : "v"(a), "v"(b));
}

// PAST: which of a row's parts lie past its width in some columns and take
// zeros there, which costs their copies an address for each lane (one row of
// 512 positions, 512 elements, 16 heads: 24.0 us with the tail so, 25.0 with
// both).
enum KwPast { KW_NONE, KW_TAIL, KW_BOTH };
constexpr int kw_ring_bytes(int DV) { return KW_RING * KW_ROWS * (DV * 2 + 128); }
template <int DK, int DV, int WQ, KwPast PAST>
__global__ __launch_bounds__(KV_NT) __attribute__((amdgpu_waves_per_eu(1, 1))) void attn_wide_kernel(AttnLaunch a)
{
    constexpr KvPart PART = KV_ALL;
    const int blk = blockIdx.x;
    __shared__ __attribute__((aligned(256))) char ring[kw_ring_bytes(DV)];
    __shared__ uint64_t rows_s[KW_BLOCK * KW_ROWS];
    __shared__ float red_m[KV_WAVES][32], red_l[KV_WAVES][32];
#include "attend_wide.h"
}

// A part of a call, a workgroup of a kernel that takes both: they have one ring.
template <int DV>
__shared__ __attribute__((aligned(256))) char kw_ring[kw_ring_bytes(DV)];
template <int DV>
__shared__ uint64_t kw_rows[KW_BLOCK * KW_ROWS];
template <int DV>
__shared__ float kw_red[2][KV_WAVES][32];
template <int DK, int DV, int WQ, KwPast PAST, KvPart PART>
__device__ __forceinline__ void attn_wide_rows(const AttnLaunch &a, int blk)
{
    auto &ring = kw_ring<DV>;
    auto &rows_s = kw_rows<DV>;
    auto &red_m = kw_red<DV>[0], &red_l = kw_red<DV>[1];
#include "attend_wide.h"
}

}  // namespace coli
