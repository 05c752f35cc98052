// attend.hip -- attention of one new token per sequence over a paged
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

// Entries of sequence b: positions, or listed ones.
__device__ __forceinline__ int kv_len(const AttnLaunch &a, int b)
{
    return a.idx ? a.idx_k : min(max(a.lens[b], 0), a.cap);
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
// sequences.
__device__ __forceinline__ void kv_prefix(const AttnLaunch &a, int b, int *before, int *total)
{
    if (a.idx) {
        const int per = kv_units(a.idx_k);
        *before = b * per;
        *total = a.B * per;
        return;
    }
    const int lane = threadIdx.x & 63;
    int lo = 0, all = 0;
    for (int i = lane; i < a.B; i += 64) {
        const int st = kv_units(kv_len(a, i));
        all += st;
        lo += (i < b) ? st : 0;
    }
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

// False: the range is empty.  R rows a sequence.  The same for every wave.
__device__ __forceinline__ bool kv_first(const AttnLaunch &a, int R, KvRange &rg)
{
    int before, total;
    kv_prefix(a, 0, &before, &total);
    total *= R;
    const int range = kv_range(a, total);
    const int u = blockIdx.x * range;         // below total + n_wg * (KV_ROW_UNITS + 1), and 2^31 by the host's check
    if (u >= total) return false;
    int base = 0;
    if (a.idx) {
        const int per = kv_units(a.idx_k) * R;
        rg.b = u / per;
        base = rg.b * per;
    } else {
        const int lane = threadIdx.x & 63;
        int sum = 0;                          // units (per row) before this chunk of sequences
        for (int c = 0;; c += 64) {
            const int st = (c + lane < a.B) ? kv_units(kv_len(a, c + lane)) : 0;
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
    rg.n = kv_len(a, rg.b);
    rg.steps = kv_steps(rg.n);
    const int per = kv_units(rg.n);
    rg.row = (u - base) / per;
    rg.s0 = (u - base) - rg.row * per;
    return true;
}

// A workgroup's range, or (direct) its row, which may be empty.
__device__ __forceinline__ bool kv_begin(const AttnLaunch &a, int R, KvRange &rg)
{
    if (!a.direct) return kv_first(a, R, rg);
    rg.b = blockIdx.x / R;
    rg.row = blockIdx.x - rg.b * R;
    rg.n = kv_len(a, rg.b);
    rg.steps = kv_steps(rg.n);
    rg.u = rg.s0 = 0;
    rg.u_end = max(rg.steps, 1);
    return true;
}

// The next row of a range (past the last sequence: one that is never taken).
__device__ __forceinline__ void kv_next_row(const AttnLaunch &a, int R, int &b, int &n, int &steps, int &row)
{
    if (++row < R) return;
    row = 0;
    do {
        ++b;
        n = b < a.B ? kv_len(a, b) : 1;
    } while (n == 0);
    steps = kv_steps(n);
}

__device__ __forceinline__ int kv_pool_row(const AttnLaunch &a, int pg, int h, int p)
{
    return (int)((((uint32_t)pg * (uint32_t)a.Hkv + (uint32_t)h) << a.page_shift) +
                 (uint32_t)(p & ((1 << a.page_shift) - 1)));
}

// Pool row of entry e < end of sequence b's positions (of its list, where
// there is one) for cache head h; -1: hidden.  No branches, and the table is
// read before the length is known: its loads wait for nothing.
__device__ __forceinline__ int kv_row(const AttnLaunch &a, int b, int h, int end, int len, int e)
{
    int p = e;
    if (a.idx) p = a.idx[(size_t)b * a.idx_k + min(e, a.idx_k - 1)];
    const int at = min(max(p, 0), a.cap - 1);
    const int pg = a.table[(size_t)b * a.max_pages + (at >> a.page_shift)];
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
template <bool BF16, int DK, int DV, int NW>
__global__ __launch_bounds__(64 * NW) void attn_kernel(AttnLaunch a)
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
    if (!kv_begin(a, R, rg)) return;
    int u = rg.u, b = rg.b, n = rg.n, steps = rg.steps, row = rg.row, s0 = rg.s0;
    const int u_begin = u, u_end = rg.u_end;

    const T *kpool = (const T *)a.k;
    const T *vpool = (const T *)(a.v ? a.v : a.k);
    const int vstride = a.v ? a.Dv : a.Dk;
    const int key_chunks = (a.Dk + 4 * EPL - 1) / (4 * EPL), full_chunks = a.Dk / (4 * EPL);

    for (; u < u_end; u += kv_units(n) - s0, s0 = 0, kv_next_row(a, R, b, n, steps, row)) {
        const int s1 = min(steps, s0 + (u_end - u));
        const int h = a.q_tiles == 1 ? row : row / a.q_tiles, q0 = (row - h * a.q_tiles) * KV_QT;
        const int nq = min(KV_QT, G - q0);    // query heads of this tile
        const size_t qrow = (size_t)b * a.Hq + h * G + q0;
        if (s0 >= steps) {                    // a row's units past its steps, or (direct) an empty row
            if (a.direct) return kv_write_empty(a, qrow, nq);
            continue;
        }
        const int len = min(max(a.lens[b], 0), a.cap);

        // the query tile: lane (j, g) holds query j's elements as a key's
        u32x4 qf[KC];
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const int d = (4 * c + g) * EPL;
            qf[c] = u32x4{0, 0, 0, 0};
            if (j < nq && d < a.Dk)
                qf[c] = *reinterpret_cast<const u32x4 *>((const T *)a.q + (qrow + j) * a.Dk + d);
        }
        f32x4 o[VC][VE];
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int e = 0; e < VE; ++e) o[c][e] = f32x4{0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, l = 0.f;

        // pool row of position `lane & 31` of step s (-1: hidden)
        const int end = min(n, s1 * KV_STEP);
        auto rows_of = [&](int s) { return kv_row(a, b, h, end, len, s * KV_STEP + (lane & 31)); };
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
            f32x4 sc[2];
            sc[0] = sc[1] = f32x4{0.f, 0.f, 0.f, 0.f};
            auto product = [&](const u32x4 &k0, const u32x4 &k1, int c) {
                if constexpr (BF16) {
                    sc[0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(k0), as_bf16(qf[c]), sc[0], 0, 0, 0);
                    sc[1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(k1), as_bf16(qf[c]), sc[1], 0, 0, 0);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[0] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k0[e]), __uint_as_float(qf[c][e]), sc[0], 0, 0, 0);
                        sc[1] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k1[e]), __uint_as_float(qf[c][e]), sc[1], 0, 0, 0);
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
            if (a.scores) {
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
        const int slot = 2 * blockIdx.x + (u == u_begin ? 0 : 1);
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
            if (whole) {
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

// Where the parts of a row are: ranges w0 .. w1 hold some of it (w0 = w1: one
// holds all, and has written the row's results); the first part's slot, the
// later ranges' being their first ones.
struct KvParts {
    int steps, w0, w1, first;
    __device__ __forceinline__ int slot(int w) const { return w == w0 ? first : 2 * w; }
};
__device__ __forceinline__ KvParts kv_parts(const AttnLaunch &a, int b, int row, int before, int total)
{
    const int R = a.Hkv * a.q_tiles, n = kv_len(a, b);
    KvParts p{kv_steps(n), 0, 0, 0};
    if (p.steps == 0) return p;
    const int range = kv_range(a, total * R);
    const int u0 = before * R + row * kv_units(n);
    p.w0 = u0 / range;
    p.w1 = (u0 + p.steps - 1) / range;
    p.first = 2 * p.w0 + (u0 == p.w0 * range ? 0 : 1);
    return p;
}

// One (sequence, query head): joins the parts that the ranges' borders left of
// it, or writes an empty sequence's zeros.  The parts are summed in the order
// of the positions.
__device__ __forceinline__ void attn_join(const AttnLaunch &a, int bq)
{
    __shared__ __attribute__((aligned(16))) float red[KV_NT * 4];
    __shared__ float factor[KV_MAX_WG];
    const int tid = threadIdx.x;
    const int b = bq / a.Hq, hq = bq - b * a.Hq;
    const int G = a.Hq / a.Hkv, h = hq / G, qi = hq - h * G, q = qi % KV_QT;
    int before, total;
    kv_prefix(a, b, &before, &total);
    const KvParts p = kv_parts(a, b, h * a.q_tiles + qi / KV_QT, before, total);
    if (p.steps == 0) return kv_write_empty(a, bq, 1);
    if (p.w0 == p.w1) return;
    auto slot_of = [&](int w) { return (size_t)p.slot(w) * KV_QT + q; };

    float mx = -INFINITY;
    for (int w = p.w0 + (tid & 63); w <= p.w1; w += 64) mx = fmaxf(mx, a.part_ml[slot_of(w) * 2]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
    const float ref = mx == -INFINITY ? 0.f : mx;
    float l = 0.f;
    for (int w = p.w0 + (tid & 63); w <= p.w1; w += 64) {
        const float f = __builtin_amdgcn_exp2f(a.part_ml[slot_of(w) * 2] - ref);
        l += a.part_ml[slot_of(w) * 2 + 1] * f;
        if (tid < 64) factor[w - p.w0] = f;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) l += __shfl_xor(l, off);
    __syncthreads();

    // groups of threads take every ng-th part, 4 columns a thread
    const int cols = a.Dv / 4, ng = KV_NT / cols, grp = tid / cols, col = tid % cols;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    if (grp < ng) {
#pragma unroll 4
        for (int w = p.w0 + grp; w <= p.w1; w += ng)
            acc += *reinterpret_cast<const f32x4 *>(a.part_o + slot_of(w) * a.Dv + 4 * col) * factor[w - p.w0];
        *reinterpret_cast<f32x4 *>(red + 4 * tid) = acc;
    }
    __syncthreads();
    if (tid < cols) {
        for (int x = 1; x < ng; ++x) acc += *reinterpret_cast<const f32x4 *>(red + 4 * (x * cols + col));
        const float inv = kv_inverse(l);
        const size_t at = (size_t)bq * a.Dv + 4 * col;
        if (a.bf16)
            *reinterpret_cast<u32x2 *>((uint16_t *)a.out + at) =
                u32x2{pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv)};
        else *reinterpret_cast<f32x4 *>((float *)a.out + at) = acc * inv;
    }
    if (tid == 0) kv_write_lse(a, bq, mx, l);
}

// Running weights of kv_weight_positions(heads) positions of a (sequence,
// cache head): acc_out = acc_in + sum over its query heads of e^(t - m) / l,
// four positions a thread.  Of many heads each wave takes a fourth, and a
// fourth of the positions (95 latent sequences of 1 to 2263 positions, 128
// heads, the whole call: 75 us with all heads a thread, 69 so).  The references m and sums l come from the row's writer or, where
// it was cut, from its parts (the wide kernel's join, which runs before,
// leaves them like a writer).
__host__ __device__ inline int kv_weight_positions(int heads) { return heads < 32 ? 4 * KV_NT : 4 * 64; }

__device__ __forceinline__ void attn_weights(const AttnLaunch &a, int at, bool joined)
{
    __shared__ float stat[KV_NT][2];
    __shared__ f32x4 others[KV_WAVES - 1][64];
    const int each = kv_weight_positions(a.Hq / a.Hkv);
    const bool split = each < 4 * KV_NT;
    const int chunks = (a.cap + each - 1) / each;
    const int tid = threadIdx.x, mine = split ? tid & 63 : tid;
    const int first = split ? tid >> 6 : 0, step = split ? KV_WAVES : 1;     // heads of the thread
    const int bh = at / chunks, b = bh / a.Hkv, h = bh - b * a.Hkv, G = a.Hq / a.Hkv;
    const int n = min(max(a.lens[b], 0), a.cap);
    const int p0 = (at - bh * chunks) * each;
    if (p0 >= n) return;
    int before = 0, total = 0;
    // the lanes that share a head's parts, as many as there may be (one sequence of 43069 positions, 7 heads: 32 us
    // with one lane a head, 10 with 32)
    int share = 1;
    if (!joined && !a.direct) {
        kv_prefix(a, b, &before, &total);
        const int most = kv_units(n) / kv_range(a, total * a.Hkv * a.q_tiles) + 2;
        while (share < most && 2 * share <= 64 && 2 * share * G <= KV_NT) share *= 2;
    }
    const int p = p0 + mine * 4;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    const int heads = KV_NT / share, sub = tid & (share - 1);
    for (int i0 = 0; i0 < G; i0 += heads) {
        const int i = i0 + tid / share;
        const size_t q = (size_t)b * a.Hq + h * G + i;
        KvParts parts{};
        if (i < G && !joined && !a.direct) parts = kv_parts(a, b, h * a.q_tiles + i / KV_QT, before, total);
        const bool cut = parts.w0 != parts.w1;
        float mx = -INFINITY, l = 0.f;
        if (cut) {                            // four parts' loads in flight
            for (int w = parts.w0 + sub; w <= parts.w1; w += 4 * share) {
                float mw[4], lw[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int at_w = w + x * share;
                    const float *ml = a.part_ml + ((size_t)parts.slot(min(at_w, parts.w1)) * KV_QT + i % KV_QT) * 2;
                    mw[x] = at_w <= parts.w1 ? ml[0] : -INFINITY;
                    lw[x] = at_w <= parts.w1 ? ml[1] : 0.f;
                }
                float mn = mx;
#pragma unroll
                for (int x = 0; x < 4; ++x) mn = fmaxf(mn, mw[x]);
                const float ref = mn == -INFINITY ? 0.f : mn;
                l *= __builtin_amdgcn_exp2f(mx - ref);
#pragma unroll
                for (int x = 0; x < 4; ++x) l += lw[x] * __builtin_amdgcn_exp2f(mw[x] - ref);
                mx = mn;
            }
        }
        for (int off = 1; off < share; off <<= 1) {
            const float mo = __shfl_xor(mx, off), lo = __shfl_xor(l, off);
            const float mn = fmaxf(mx, mo), ref = mn == -INFINITY ? 0.f : mn;
            l = l * __builtin_amdgcn_exp2f(mx - ref) + lo * __builtin_amdgcn_exp2f(mo - ref);
            mx = mn;
        }
        if (i < G && sub == 0) {
            stat[tid / share][0] = cut ? (mx == -INFINITY ? 0.f : mx) : a.stats[2 * q];
            stat[tid / share][1] = cut ? kv_inverse(l) : a.stats[2 * q + 1];
        }
        __syncthreads();
        if (p < n) {
#pragma unroll 8
            for (int i = i0 + first; i < min(G, i0 + heads); i += step) {
                const f32x4 t =
                    *reinterpret_cast<const f32x4 *>(a.scores + ((size_t)b * a.Hq + h * G + i) * a.s_ld + p);
                const float m = stat[i - i0][0], inv = stat[i - i0][1];
#pragma unroll
                for (int x = 0; x < 4; ++x) sum[x] += __builtin_amdgcn_exp2f(t[x] - m) * inv;
            }
        }
        __syncthreads();
    }
    if (split) {
        if (first > 0) others[first - 1][mine] = sum;
        __syncthreads();
        if (first > 0) return;
#pragma unroll
        for (int w = 0; w < KV_WAVES - 1; ++w) sum += others[w][mine];
    }
    if (p >= n) return;
    const size_t to = (size_t)bh * a.ld + p;
    if (p + 4 <= n) {
        if (a.acc_in) sum += *reinterpret_cast<const f32x4 *>(a.acc_in + to);
        *reinterpret_cast<f32x4 *>(a.acc_out + to) = sum;
    } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (p + x < n) a.acc_out[to + x] = sum[x] + (a.acc_in ? a.acc_in[to + x] : 0.f);
    }
}

// What follows the main kernel, in one launch: n_join workgroups join, the
// others keep the running weights.
__global__ __launch_bounds__(KV_NT) void attn_finish_kernel(AttnLaunch a, int n_join, bool joined)
{
    if ((int)blockIdx.x < n_join) attn_join(a, blockIdx.x);
    else attn_weights(a, blockIdx.x - n_join, joined);
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
template <int DK, int DV, int WQ, KwPast PAST>
__global__ __launch_bounds__(KV_NT) __attribute__((amdgpu_waves_per_eu(1, 1))) void attn_wide_kernel(AttnLaunch a)
{
    constexpr int WK = KV_WAVES / WQ;
    constexpr int RA = DV / 8;                // chunks of a row's first part
    static_assert((RA == 64 || RA == 32) && DK == DV + 64, "row parts");
    constexpr int RPC = 64 / RA;              // rows of a copy instruction
    constexpr int FIRST = KW_ROWS * RA * 16;  // bytes of a stage's first part
    constexpr int STAGE = FIRST + KW_ROWS * 128;
    constexpr int CA = KW_ROWS / RPC, CB = 4; // copy instructions of a stage's parts
    constexpr int SHARE = WQ == 1 ? 1 : KV_WAVES;         // waves that bring a stage (WQ = 1: each its own)
    constexpr int CPW = (CA + CB) / SHARE;    // copies of a wave
    constexpr int AHEAD = KW_RING / WK - 1;   // rounds in flight beside the one computed
    constexpr int KS = DK / 16, DT = DV / 32;
    static_assert(KS % 4 == 0, "fragments in fours");
    constexpr int OUT = 32 * DV;              // floats of a query tile's output
    static_assert(KV_WAVES * OUT * 2 <= KW_RING * STAGE, "half of each wave's output fits the ring");
    __shared__ __attribute__((aligned(256))) char ring[KW_RING * STAGE];
    __shared__ uint64_t rows_s[KW_BLOCK * KW_ROWS];         // addresses of the stages' rows
    __shared__ float red_m[KV_WAVES][32], red_l[KV_WAVES][32];

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);    // uniform: the copies' LDS addresses are
    const int qt = wave % WQ, kb = wave / WQ;
    const int G = a.Hq / a.Hkv;
    const int R = a.Hkv * a.q_tiles;
    KvRange rg;
    if (!kv_first(a, R, rg)) return;
    int u = rg.u, b = rg.b, n = rg.n, steps = rg.steps, row = rg.row, s0 = rg.s0;
    const int u_begin = u, u_end = rg.u_end;
    const char *pool = (const char *)a.k;
    const int row_bytes = PAST == KW_NONE ? DK * 2 : a.Dk * 2;
    const uint32_t ring_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)ring;

    float known = -INFINITY;                  // the reference of a row that is run again
    bool again = false;
    auto advance = [&] {
        u += kv_units(n) - s0;
        s0 = 0;
        kv_next_row(a, R, b, n, steps, row);
    };
    for (; u < u_end; again ? (void)0 : advance()) {
        const int s1 = min(steps, s0 + (u_end - u));
        if (s0 >= steps) continue;            // a row's units past its steps
        // The lane number is made opaque here (and in issue): the offsets that
        // follow from it are cheap to form again, and kept over the whole row
        // loop they would push the operands out of the registers.
        int lane = tid & 63;
        asm volatile("" : "+v"(lane));
        const int ql = lane & 31, hi = lane >> 5;
        // This lane's places inside a stage, as bytes: key row ql, chunks hi and
        // RA + hi (chunk c of the row: XOR by 16 times c's even part, low four or
        // three bits), and the transposing reads' (below).
        const int key_at = ql * (RA * 16) + ((hi ^ kw_swz(ql)) << 4);
        const int tail_at = FIRST + ql * 128 + ((hi ^ ((ql >> 1) & 7)) << 4);
        // A transposing read takes rows 16 ks + 8 half + 4 hi + 0..3 (16 lanes: 4 rows of 32 bytes): this is for
        // ks = half = 0 and column 16 * (bit 4 of the lane).
        const int rr = (lane & 15) >> 2;
        const int val_at = (4 * hi + rr) * (RA * 16) + (((2 * ((lane >> 4) & 1) + ((lane >> 1) & 1)) ^ (rr << 2) ^ hi) << 4) +
                           (lane & 1) * 8;
        const int h = row / a.q_tiles, q0 = (row % a.q_tiles) * (32 * WQ) + 32 * qt;
        const int nq = G - q0;                // query heads of this wave's tile (may be none)
        const size_t qrow = (size_t)b * a.Hq + h * G + q0;
        const int len = min(max(a.lens[b], 0), a.cap);
        const int seg = s1 - s0, rounds = (seg + WK - 1) / WK;

        f32x16 o[DT];
        float m = known, l, top;              // m: the reference; top: the largest score

        // row addresses of the block of stages that holds stage t0 (a multiple of KW_BLOCK)
        auto look_up = [&](int t0) {
            constexpr int PER = KW_BLOCK * KW_ROWS / KV_NT;
            const int first = (s0 + t0) * KV_STEP + tid, end = min(n, s1 * KV_STEP);
            int p[PER];
#pragma unroll
            for (int x = 0; x < PER; ++x) {   // no branches: all loads of a kind in flight together
                const int e = first + x * KV_NT;
                p[x] = a.idx ? a.idx[(size_t)b * a.idx_k + min(e, n - 1)] : e;
                p[x] = (e < end && p[x] >= 0 && p[x] < len) ? p[x] : -1;
            }
            int pg[PER];
#pragma unroll
            for (int x = 0; x < PER; ++x) pg[x] = a.table[(size_t)b * a.max_pages + (max(p[x], 0) >> a.page_shift)];
#pragma unroll
            for (int x = 0; x < PER; ++x)
                rows_s[tid + x * KV_NT] =
                    (p[x] >= 0 && pg[x] >= 0 && pg[x] < a.n_pages)
                        ? (uint64_t)pool + (uint64_t)(uint32_t)kv_pool_row(a, pg[x], h, p[x]) * (uint32_t)row_bytes
                        : (uint64_t)kv_zeros;
        };
        // Copy instructions of 32 rows' two parts into the stage at byte dst; rows: lane i holds row i's address.
        // Columns past the row's width are zeros.
        const uint32_t last = row_bytes - 16;
        auto first_off = [&](int i) {                       // the lane's place in its row
            uint32_t lane_at = (lane & (RA - 1)) << 4;
            if constexpr (RPC == 2) lane_at ^= (lane >> 5) << 6;
            return lane_at ^ (kw_swz(i * RPC) << 4);
        };
        auto tail_off = [&](int i) { return (uint32_t)(RA + ((lane & 7) ^ ((4 * i + (lane >> 4)) & 7))) << 4; };
        auto inside = [&](uint64_t src, uint32_t off) { return (off <= last ? src : (uint64_t)kv_zeros) + off; };
        auto copy_first = [&](uint64_t rows, int i, uint32_t dst) {
            const uint32_t off = first_off(i);
            const uint64_t src = kw_lane(rows, i * RPC);
            if constexpr (RPC == 1) {
                if constexpr (PAST == KW_BOTH) kw_copy(inside(src, off), dst + i * 1024);
                else kw_copy(src, off, dst + i * 1024);
            } else {
                const uint64_t other = kw_lane(rows, i * RPC + 1), mine = lane < 32 ? src : other;
                kw_copy(PAST == KW_BOTH ? inside(mine, off) : mine + off, dst + i * 1024);
            }
        };
        auto copy_tail = [&](uint64_t rows, int i, uint32_t dst) {
            const uint64_t src = (uint64_t)__shfl((unsigned long long)rows, 8 * i + (lane >> 3));
            kw_copy(PAST == KW_NONE ? src + tail_off(i) : inside(src, tail_off(i)), dst + FIRST + i * 1024);
        };
        // copy number i of the wave's share of stage t
        auto copy = [&](int t, uint64_t rows, int i) {
            const uint32_t dst = ring_at + (t % KW_RING) * STAGE;
            const int me = SHARE == 1 ? 0 : wave;
            if (i < CA / SHARE) copy_first(rows, i * SHARE + me, dst);
            else copy_tail(rows, (i - CA / SHARE) * SHARE + me, dst);
        };
        // lane i's: address of row i (lane 32 + i: the same) of stage t, and which rows are hidden
        auto stage_rows = [&](int t) { return rows_s[(t % KW_BLOCK) * KW_ROWS + ql]; };
        auto hidden = [&](uint64_t rows) { return (uint32_t)__ballot(rows == (uint64_t)kv_zeros); };
        auto issue = [&](int t) {
            const uint64_t rows = stage_rows(t);
#pragma unroll 4
            for (int i = 0; i < CPW; ++i) copy(t, rows, i);
            return hidden(rows);
        };

        // Query fragments and key fragments are the same places of a stage: group grp of four, number x of it, is
        // columns 16 frag(grp, x) + 8 hi + 0..7; the last group is the tail.
        constexpr int GRP = KS / 4;
        auto frag = [](int grp, int x) {
            return grp == GRP - 1 ? RA / 2 + x : RA == 64 ? grp + 8 * x : 2 * grp + (x >> 1) + 8 * (x & 1);
        };
        auto frag_at = [&](const char *st, int grp, int x) {
            const int c = frag(grp, x);
            const int at = grp == GRP - 1 ? tail_at ^ (32 * x) : (key_at ^ (32 * (c & 7))) + (c >> 3) * 256;
            return *reinterpret_cast<const bf16x8 *>(st + at);
        };

        // The queries come in like a stage, each tile by its waves, zeros past their width, and stay in registers as the
        // score operand.
        bf16x8 qf[KS];
        {
            const uint64_t rows = ql < nq ? (uint64_t)a.q + (qrow + ql) * row_bytes : (uint64_t)kv_zeros;
            const uint32_t dst = ring_at + qt * STAGE;
            auto bring = [&](int r, uint32_t off, uint32_t to) {
                const uint64_t src = (uint64_t)__shfl((unsigned long long)rows, r);
                kw_copy(inside(src, off), to);
            };
#pragma unroll 1
            for (int i = kb; i < CA; i += WK) bring(i * RPC + (RPC == 1 ? 0 : lane >> 5), first_off(i), dst + i * 1024);
#pragma unroll 1
            for (int i = kb; i < CB; i += WK) bring(8 * i + (lane >> 3), tail_off(i), dst + FIRST + i * 1024);
            look_up(0);
            kw_wait_copies<0>();
            kw_barrier();
#pragma unroll
            for (int c = 0; c < KS; ++c) qf[c] = frag_at(ring + qt * STAGE, c / 4, c % 4);
            kw_barrier();
        }

        // The reference is the largest score of the wave's first stage and stays:
        // weights are numbers of fp32's and bf16's whole range, so a later score
        // may pass it by up to 2^60 without harm, and O^T never has to be moved to
        // another one.  A row where some score passes it further is run again with
        // its largest score as the reference, by all waves (they share the stages),
        // and so is one where large values have met weights past 2^20 and a sum is
        // no number.
        float above;
        bool far;
        for (;;) {
            l = 0.f;
            top = -INFINITY;
#pragma unroll
            for (int t = 0; t < DT; ++t) {
                // zero by a product: one instruction for sixteen registers (256 writes were 2 KB of code)
                o[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf16x8{}, bf16x8{}, f32x16{}, 0, 0, 0);
                asm volatile("" : "+a"(o[t]));    // at home in the accumulation registers
            }
            uint32_t hids[AHEAD + 1];                       // hidden rows of the wave's stages in flight, next one first
            if constexpr (AHEAD > 0) {
#pragma unroll 1
                for (int t = 0; t < AHEAD * WK; ++t) {
                    const uint32_t mask = issue(t);
#pragma unroll
                    for (int y = 0; y < AHEAD; ++y)
                        if (t == y * WK + kb) hids[y] = mask;
                }
            }
            for (int r = 0; r < rounds; ++r) {
                const int ahead = (r + AHEAD) * WK;         // first stage of the round to be copied in this one
                if constexpr (AHEAD > 0) {
                    // this wave's copies of round r have landed, then everyone's; round r - 1 is done with its stages
                    kw_wait_copies<(AHEAD - 1) * WK * CPW>();
                    kw_barrier();
                    if (ahead % KW_BLOCK == 0) {
                        look_up(ahead);
                        kw_barrier();
                    }
                } else {
                    // a stage of the wave's own: the other three waves' work covers its copies
                    if (r > 0 && r * WK % KW_BLOCK == 0) {
                        kw_barrier();
                        look_up(r * WK);
                        kw_barrier();
                    }
                    hids[0] = issue(r * WK + kb);
                    kw_wait_copies<0>();
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                }
                const int t = r * WK + kb;
                // A wave without positions (t >= seg: all of them hidden) or queries (nq <= 0: zeros) computes all the
                // same: a second way through the loop would cost the accumulators their registers.
                const char *st = ring + (t % KW_RING) * STAGE;
                const uint32_t hid = hids[0] >> (4 * hi);

                // ---- scores, with the copies of a later round between the products (a wave that issues them in one
                // go multiplies nothing meanwhile: 2000 cycles of 7200) ----
                f32x16 sc;
                {
                    // Eight fragments in a ring: the one just used makes room for the one eight products on (the order is
                    // fixed: left to itself the compiler reads all 36 ahead and spills).
#pragma unroll
                    for (int i = 0; i < 16; ++i) sc[i] = 0.f;
                    static_assert(AHEAD == 0 || CPW == GRP, "a copy of each stage to a group");
                    bf16x8 kf[8];
                    uint64_t rows[WK];
#pragma unroll
                    for (int x = 0; x < 8; ++x) kf[x] = frag_at(st, x / 4, x % 4);
                    if constexpr (AHEAD > 0) {
#pragma unroll
                        for (int y = 0; y < WK; ++y) rows[y] = stage_rows(ahead + y);
#pragma unroll
                        for (int y = 0; y < AHEAD; ++y) hids[y] = hids[y + 1];
#pragma unroll
                        for (int y = 0; y < WK; ++y)
                            if (y == kb) hids[AHEAD - 1] = hidden(rows[y]);
                    }
#pragma unroll
                    for (int grp = 0; grp < GRP; ++grp) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {       // a read after each product: the four waves share the LDS port
                            kw_mfma_v(sc, kf[(4 * grp + x) % 8], qf[4 * grp + x]);
                            if (grp + 2 < GRP) kf[(4 * grp + x) % 8] = frag_at(st, grp + 2, x);
                            if constexpr (AHEAD > 0) {
                                if (x % 2 == 1 && x / 2 < WK) copy(ahead + x / 2, rows[x / 2], grp);
                            }
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                    // the last product's result: 18 cycles of wait states before a vector instruction may read it
                    asm volatile("s_nop 15\n\ts_nop 7" : "+v"(sc));
                }
                // ---- weights: query ql, position 8 (i >> 2) + 4 hi + (i & 3) ----
                float w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = kv_scaled(a, sc[i]);
                if (__ballot(hid != 0)) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (hid >> (8 * (i >> 2) + (i & 3)) & 1) w[i] = -INFINITY;
                }
                if (a.scores && ql < nq && t < seg) {
                    float *dst = a.scores + (qrow + ql) * a.s_ld + (s0 + t) * KV_STEP + 4 * hi;
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        *reinterpret_cast<f32x4 *>(dst + 8 * x) = f32x4{w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]};
                }
                float mx = w[0];
#pragma unroll
                for (int i = 1; i < 16; ++i) mx = fmaxf(mx, w[i]);
                top = fmaxf(top, mx);
                if (__ballot(m == -INFINITY)) {             // nothing seen yet
                    mx = fmaxf(mx, __shfl_xor(mx, 32));
                    m = m == -INFINITY ? mx : m;
                }
                const float ref = (m == -INFINITY) ? 0.f : m;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    w[i] = __builtin_amdgcn_exp2f(w[i] - ref);
                    l += w[i];
                }
                u32x4 whi[2], wlo[2];
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float a0 = w[8 * ks + 2 * x], a1 = w[8 * ks + 2 * x + 1];
                        whi[ks][x] = pack_bf16(a0, a1);
                        wlo[ks][x] = pack_bf16(a0 - __uint_as_float(whi[ks][x] << 16),
                                               a1 - __uint_as_float(whi[ks][x] & 0xffff0000u));
                    }
                // ---- output: slots 0-3 of a lane are positions 16 ks + 4 hi + 0..3, slots 4-7 the ones 8 further ----
                // two column tiles at a time, read one pair ahead, their products taken in turn
                s16x4 vf[2][2][2][2];
                auto column = [&](int x, int y) {           // read number y of eight: columns 64 x .. + 63
                    const int odd = y & 1, half = (y >> 1) & 1, ks = y >> 2;
                    const int at = (val_at ^ ((x & 1) * 128 + odd * 64 + half * 32)) + (x >> 1) * 256 +
                                   (16 * ks + 8 * half) * (RA * 16);
                    vf[x & 1][odd][ks][half] =
                        __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(st + at));
                };
#pragma unroll
                for (int y = 0; y < 8; ++y) column(0, y);
#pragma unroll
                for (int x = 0; x < DT / 2; ++x) {
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const int odd = y & 1, ks = y >> 2;
                        const bf16x8 vb = __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(
                            vf[x & 1][odd][ks][0], vf[x & 1][odd][ks][1], 0, 1, 2, 3, 4, 5, 6, 7));
                        o[2 * x + odd] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vb, as_bf16((y & 2) ? wlo[ks] : whi[ks]),
                                                                                o[2 * x + odd], 0, 0, 0);
                        if (x + 1 < DT / 2) column(x + 1, y);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    asm volatile("" : "+a"(o[2 * x]), "+a"(o[2 * x + 1]));
                }
            }
            kw_wait_copies<0>();                            // stages past the row's end are copied too, as zeros
            top = fmaxf(top, __shfl_xor(top, 32));
            above = top - m;                                // (no number where nothing was seen: not above anything)
            far = __syncthreads_or(above > 20.f);
            if (!far || !__syncthreads_or(above > 60.f)) break;
            m = top;
            look_up(0);
            kw_barrier();
        }

        // ---- the waves of a query tile become one (the ring is free: its copies have landed and been read) ----
        l += __shfl_xor(l, 32);
        if (hi == 0) {
            red_m[wave][ql] = m;
            red_l[wave][ql] = l;
        }
        kw_barrier();
        float ma = m, la = l, f[WK];
        if constexpr (WK > 1) {
            ma = red_m[qt][ql];
#pragma unroll
            for (int w = 1; w < WK; ++w) ma = fmaxf(ma, red_m[w * WQ + qt][ql]);
            la = 0.f;
#pragma unroll
            for (int w = 0; w < WK; ++w) {
                const float mw = red_m[w * WQ + qt][ql];
                f[w] = mw == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mw - ma);
                la += red_l[w * WQ + qt][ql] * f[w];
            }
        }
        // columns 32 x + 8 i + 4 hi .. + 3 of query ql go out
        const bool whole = s0 == 0 && s1 == steps;
        const float inv = kv_inverse(la);
        const size_t slot = (size_t)(2 * blockIdx.x + (u == u_begin ? 0 : 1)) * WQ + qt;
        f32x4 *part = reinterpret_cast<f32x4 *>(a.part_o + slot * OUT) + lane;
        uint16_t *out = (uint16_t *)a.out + (qrow + ql) * a.Dv;
        auto put = [&](int x, int i, f32x4 v) {
            if (!whole) {                     // a part: lanes side by side (attn_wide_join_kernel reads it the same way)
                part[(x * 4 + i) * 64] = v;
            } else if (ql < nq && 32 * x + 8 * i + 4 * hi < a.Dv) {  // Dv is a multiple of 8: all four columns or none
                *reinterpret_cast<u32x2 *>(out + 32 * x + 8 * i + 4 * hi) =
                    u32x2{pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv)};
            }
        };
        if constexpr (WK == 1) {
            if (nq > 0) {
#pragma unroll
                for (int x = 0; x < DT; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        put(x, i, f32x4{o[x][4 * i], o[x][4 * i + 1], o[x][4 * i + 2], o[x][4 * i + 3]});
                        __builtin_amdgcn_sched_barrier(0);
                    }
            }
        } else {
            // Half of the tile's columns at a time, all waves' side by side in LDS; each wave sums its share of them.
            // (Exchanges of halves between pairs of waves move less, but are five times the code.)
            f32x4 *buf = reinterpret_cast<f32x4 *>(ring);
            constexpr int H = DT / 2;
            auto give = [&](auto half) {
#pragma unroll
                for (int x = 0; x < H; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x16 &t = o[decltype(half)::value * H + x];
                        buf[((wave * H + x) * 4 + i) * 64 + lane] =
                            f32x4{t[4 * i], t[4 * i + 1], t[4 * i + 2], t[4 * i + 3]};
                    }
            };
#pragma unroll 1
            for (int p = 0; p < 2; ++p) {
                if (p == 0) {
                    give(KwInt<0>{});
                } else {
                    kw_barrier();
                    give(KwInt<1>{});
                }
                kw_barrier();
                if (nq > 0) {
#pragma unroll 1
                    for (int y = kb; y < H; y += WK) {
                        f32x4 v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            v[i] = buf[((qt * H + y) * 4 + i) * 64 + lane] * f[0];
#pragma unroll
                            for (int w = 1; w < WK; ++w) v[i] += buf[(((w * WQ + qt) * H + y) * 4 + i) * 64 + lane] * f[w];
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) put(p * H + y, i, v[i]);
                    }
                }
            }
        }
        if (nq > 0 && kb == 0 && hi == 0) {
            if (!whole) {
                a.part_ml[(slot * 32 + ql) * 2] = ma;
                a.part_ml[(slot * 32 + ql) * 2 + 1] = la;
            } else if (ql < nq) {
                kv_write_stats(a, qrow + ql, ma, la);
            }
        }
        again = false;
        if (far) {
            // Weights of up to 2^60 may have taken sums past fp32's end: what this wave wrote is read back, and a row with
            // no number among it is run again (its references are its largest scores then: `far` is false).
            bool bad = false;
            if (ql < nq) {
#pragma unroll 1
                for (int x = 0; x < DT; ++x) {
                    if (WK > 1 && x % (DT / 2) % WK != kb) continue;
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        if (!whole) {
                            const f32x4 v = part[(x * 4 + i) * 64];
#pragma unroll
                            for (int c = 0; c < 4; ++c) bad |= !(fabsf(v[c]) < INFINITY);
                        } else if (32 * x + 8 * i + 4 * hi < a.Dv) {
                            const u32x2 v = *reinterpret_cast<const u32x2 *>(out + 32 * x + 8 * i + 4 * hi);
#pragma unroll
                            for (int c = 0; c < 2; ++c) bad |= (v[c] & 0x7f80u) == 0x7f80u || (v[c] & 0x7f800000u) == 0x7f800000u;
                        }
                    }
                }
            }
            again = __syncthreads_or(bad);
        }
        kw_barrier();                                       // red_m, red_l and the ring are free again
        known = again ? top : -INFINITY;
    }
}

// Joins the parts that attn_wide_kernel left: a workgroup takes COLS
// 32-column tiles of one query tile's output, a thread 4 columns of a query
// in each.  NG groups of threads take every NG-th part and are summed in their
// order.
template <int DV, int WQ, int COLS, int NG>
__global__ __launch_bounds__(KV_NT * NG) void attn_wide_join_kernel(AttnLaunch a)
{
    constexpr int SPLIT = DV / 32 / COLS, NF = KV_NT * NG / 32;
    __shared__ float factor[KW_MAX_WG][32], red[NF][32];
    __shared__ f32x4 others[NG > 1 ? NG - 1 : 1][NG > 1 ? COLS : 1][NG > 1 ? KV_NT : 1];
    const int tid = threadIdx.x % KV_NT, ng = threadIdx.x / KV_NT, lane = tid & 63, wave = tid >> 6;
    const int ql = lane & 31, hi = lane >> 5;
    int at = blockIdx.x;
    const int part = at % SPLIT;
    at /= SPLIT;
    const int qt = at % WQ;
    at /= WQ;
    const int R = a.Hkv * a.q_tiles, row = at % R, b = at / R;
    const int G = a.Hq / a.Hkv, h = row / a.q_tiles, q0 = (row % a.q_tiles) * (32 * WQ) + 32 * qt;
    const int nq = G - q0;
    if (nq <= 0) return;
    int before, total;
    kv_prefix(a, b, &before, &total);
    const KvParts p = kv_parts(a, b, row, before, total);
    const size_t q = (size_t)b * a.Hq + h * G + q0 + ql;
    uint16_t *out = (uint16_t *)a.out + q * a.Dv;
    // wave i of the workgroup holds the i-th 8 columns of each tile: its lanes' are 8 i + 4 hi + 0..3
    f32x4 sum[COLS];
#pragma unroll
    for (int x = 0; x < COLS; ++x) sum[x] = f32x4{0.f, 0.f, 0.f, 0.f};
    float mx = -INFINITY, l = 0.f;
    if (p.steps > 0) {
        if (p.w0 == p.w1) return;                           // one range holds all of it
        auto slot_of = [&](int w) { return (size_t)p.slot(w) * WQ + qt; };
        // the parts' factors for the 32 queries: the workgroup's NF groups of 32 threads take every NF-th part
        const int grp = threadIdx.x >> 5;
        for (int w = p.w0 + grp; w <= p.w1; w += NF) mx = fmaxf(mx, a.part_ml[(slot_of(w) * 32 + ql) * 2]);
        red[grp][ql] = mx;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < NF; ++x) mx = fmaxf(mx, red[x][ql]);
        const float ref = mx == -INFINITY ? 0.f : mx;
        for (int w = p.w0 + grp; w <= p.w1; w += NF) {
            const float f = __builtin_amdgcn_exp2f(a.part_ml[(slot_of(w) * 32 + ql) * 2] - ref);
            l += a.part_ml[(slot_of(w) * 32 + ql) * 2 + 1] * f;
            factor[w - p.w0][ql] = f;
        }
        __syncthreads();
        red[grp][ql] = l;
        __syncthreads();
        l = 0.f;
#pragma unroll
        for (int x = 0; x < NF; ++x) l += red[x][ql];
#pragma unroll 16 / COLS
        for (int w = p.w0 + ng; w <= p.w1; w += NG) {
            const f32x4 *src = reinterpret_cast<const f32x4 *>(a.part_o + slot_of(w) * (32 * DV)) + lane;
            const float f = factor[w - p.w0][ql];
#pragma unroll
            for (int x = 0; x < COLS; ++x) sum[x] += src[((part * COLS + x) * 4 + wave) * 64] * f;
        }
        if constexpr (NG > 1) {
            if (ng > 0) {
#pragma unroll
                for (int x = 0; x < COLS; ++x) others[ng - 1][x][tid] = sum[x];
            }
            __syncthreads();
            if (ng == 0) {
#pragma unroll
                for (int y = 0; y < NG - 1; ++y)
#pragma unroll
                    for (int x = 0; x < COLS; ++x) sum[x] += others[y][x][tid];
            }
        }
    }
    if (ng > 0 || ql >= nq) return;
    const float inv = kv_inverse(l);
#pragma unroll
    for (int x = 0; x < COLS; ++x) {
        const int d = 32 * (part * COLS + x) + 8 * wave + 4 * hi;
        if (d < a.Dv)
            *reinterpret_cast<u32x2 *>(out + d) = u32x2{pack_bf16(sum[x][0] * inv, sum[x][1] * inv),
                                                        pack_bf16(sum[x][2] * inv, sum[x][3] * inv)};
    }
    if (part == 0 && wave == 0 && hi == 0) kv_write_stats(a, q, mx, l);
}

// How a call runs.  entries: the longest row there may be (the table's room, or
// the listed positions): the lengths are on the device.  Short sequences in
// wide tables are cut like long ones (64 sequences of 1 to 200 positions, 32 /
// 8 heads of 128: 9.3 us in tables for 224 positions, 14.4 for 1792 or 14336;
// with running weights 13.7, 19.8, 25.5, by the second pass's grid).
AttnPlan attn_plan(int B, int Hq, int Hkv, int Dk, int Dv, bool bf16, bool latent, int entries)
{
    AttnPlan p{};
    const int G = Hq / Hkv, d = Dk > Dv ? Dk : Dv;
    const int steps = (entries + KV_STEP - 1) / KV_STEP;
    // bf16 rows past 256 elements (latent caches by the host's check) take the
    // LDS kernel, and latent rows past 128 where several query tiles would
    // read much of them each (256 elements, us there / in the LDS kernel: 32
    // sequences of 4096 positions with 16 heads 33.6 / 34.5, 32 heads 47 / 35,
    // 128 heads 134 / 54; of 1024 with 32 heads 23.7 / 20.7; 8 of 512 with 32
    // heads 16.4 / 17.9, with 128 22.2 / 19.4).
    const long work = (long)B * Hkv * steps;
    p.wide = bf16 && (Dk > 256 || (latent && Dk > 128 && G > KV_QT && work * ((G + KV_QT - 1) / KV_QT) >= 8 * KW_MAX_WG));
    if (p.wide) {
        // Fewer tiles a workgroup: more workgroups for small work, which then
        // read the cache (out of the caches) more often.  128 heads, us with
        // 1 / 2 / 4: one row of 512 positions 23.6 / 28.5 / 37.2, 8 of 2048
        // 32.6 / 35.2 / 44.2, 32 of 1024 51.5 / 46.1 / 51.9, 64 of 2048
        // 113 / 86 / 93, 64 of 8192 358 / 252 / 241; 64 heads, 1 / 2: one row
        // of 512 23.8 / 28.7, 8 of 2048 29.3 / 33.3, 64 of 2048 77 / 66.
        p.wq = G <= 32 || work <= 2 * KW_MAX_WG ? 1 : G <= 64 || work <= 32 * KW_MAX_WG ? 2 : 4;
        p.tile_rows = 32 * p.wq;
        p.out_cols = (Dk <= 320 && Dv <= 256) ? 256 : 512;
        p.n_wg = KW_MAX_WG;
    } else {
        p.tile_rows = KV_QT;
        p.out_cols = Dv;
        // As many as the registers let run at once: with 256 more, 128
        // sequences of 4096 positions (8 of 32 heads) take 210 -> 272 us at
        // width 64, 382 -> 446 at 128; 65536 positions alone 95 -> 112 at 256;
        // with 256 less 62 -> 69 us (width 64, one sequence of 65536).
        // (fp32 width 192, 32 sequences of 4096 positions, 8 heads: 288 us, 297
        // in the 256-wide kernel; bf16 150 in both)
        p.tier = d <= 64 ? 64 : d <= 128 ? 128 : d <= 192 && !bf16 ? 192 : d <= 256 ? 256 : (d <= 320 && Dv <= 256) ? 320 : 512;
        p.n_wg = 256 * (d <= (bf16 ? 128 : 64) ? 2 : 1);
    }
    p.q_tiles = (G + p.tile_rows - 1) / p.tile_rows;
    p.min_units = p.wide ? KV_ROW_UNITS : 4;
    // Short rows: a workgroup each, and no join.  A workgroup's waves: those
    // that give the fewest rounds of resident workgroups times a row's steps
    // one after the other, 2.5 more for its start and end (us, measured with
    // 1 / 2 / 4 waves: bf16 width 128, 1024 rows of 20 positions 7.8 / 8.0 /
    // 12.4, of 250 33 / 31 / 34, 1152 of 250 36 / 41 / 39; fp32 width 192, 512
    // rows of 128 positions 65 / 47 / 57, 1024 of 250 142 / 155 / 174; with
    // 4 / 8 bf16 width 128, 256 rows of 1024 33.1 / 30.0, 320 of them 41.9 /
    // 45.7).  Fewer waves have to be a fifth cheaper: they leave a long row
    // among short ones to itself (760 rows of up to 575 positions, width 192:
    // 47 us with four, 57 with one).
    const long rows = (long)B * Hkv * p.q_tiles;
    const bool light = d <= (bf16 ? 128 : 64);              // two waves a SIMD
    p.waves = KV_WAVES;
    if (!p.wide && d <= 256) {
        float best = INFINITY;
        for (int nw = light ? 8 : 4; nw >= 1; nw /= 2) {
            const long rounds = (rows * nw + 255) / 256;    // of all CUs' waves: 8 or 4 each
            const float cost = (float)((rounds + (light ? 7 : 3)) / (light ? 8 : 4)) * (2.5f + (float)((steps + nw - 1) / nw));
            if (cost < 0.8f * best) best = cost, p.waves = nw;
        }
    }
    // How long a row may be goes by the steps a wave takes, which many rows
    // cover and few do not (whole against cut, 8 cache heads of width 128: 1
    // sequence of 512 positions 9.8 / 10.8, of 1024 14.1 / 11.7; 8 of 1024
    // 16.0 / 15.7; 24 of 1024 25.0 / 31.5; 32 of 2048 53.6 / 61, but there
    // lengths that differ would leave most CUs waiting).
    p.direct = !p.wide && steps <= 32 && (rows >= 192 || steps <= p.waves * (rows < 64 ? 2 : 4));
    if (p.direct) p.n_wg = (int)rows;
    else p.waves = KV_WAVES;
    return p;
}

template <bool BF16, int DK, int DV>
static void launch_tier(const AttnLaunch &a, int waves, hipStream_t st)
{
    if constexpr (DK <= 256) {
        if (waves == 1) return attn_kernel<BF16, DK, DV, 1><<<a.n_wg, 64, 0, st>>>(a);
        if (waves == 2) return attn_kernel<BF16, DK, DV, 2><<<a.n_wg, 128, 0, st>>>(a);
    }
    if constexpr (DK <= (BF16 ? 128 : 64)) {
        if (waves == 8) return attn_kernel<BF16, DK, DV, 8><<<a.n_wg, 512, 0, st>>>(a);
    }
    attn_kernel<BF16, DK, DV, KV_WAVES><<<a.n_wg, KV_NT, 0, st>>>(a);
}

template <bool BF16>
static void launch_main(const AttnLaunch &a, const AttnPlan &p, hipStream_t st)
{
    if (p.tier == 64) launch_tier<BF16, 64, 64>(a, p.waves, st);
    else if (p.tier == 128) launch_tier<BF16, 128, 128>(a, p.waves, st);
    else if (p.tier == 256) launch_tier<BF16, 256, 256>(a, p.waves, st);
    else if constexpr (!BF16) {
        if (p.tier == 192) launch_tier<BF16, 192, 192>(a, p.waves, st);
        else if (p.tier == 320) launch_tier<BF16, 320, 256>(a, p.waves, st);
        else launch_tier<BF16, 576, 512>(a, p.waves, st);
    }
}

template <int DK, int DV, int WQ>
static void launch_wide(const AttnLaunch &a, hipStream_t st)
{
    if (a.Dk == DK) attn_wide_kernel<DK, DV, WQ, KW_NONE><<<a.n_wg, KV_NT, 0, st>>>(a);
    else if (a.Dk >= DV) attn_wide_kernel<DK, DV, WQ, KW_TAIL><<<a.n_wg, KV_NT, 0, st>>>(a);
    else attn_wide_kernel<DK, DV, WQ, KW_BOTH><<<a.n_wg, KV_NT, 0, st>>>(a);
    // Of few rows the parts are many and the tiles few: more threads for each
    // (64 heads, whole calls, us with 256 / 1024 threads: one row of 32768
    // positions 60 / 44, 4 of 32768 69 / 65, 16 of 2048 38 / 42).
    const int tiles = a.B * a.Hkv * a.q_tiles * WQ * (DV / 32);
    if (tiles <= KW_MAX_WG) attn_wide_join_kernel<DV, WQ, 1, 4><<<tiles, 4 * KV_NT, 0, st>>>(a);
    else attn_wide_join_kernel<DV, WQ, 4, 1><<<tiles / 4, KV_NT, 0, st>>>(a);
}

template <int DK, int DV>
static void launch_wide(const AttnLaunch &a, int wq, hipStream_t st)
{
    if (wq == 1) launch_wide<DK, DV, 1>(a, st);
    else if (wq == 2) launch_wide<DK, DV, 2>(a, st);
    else launch_wide<DK, DV, 4>(a, st);
}

hipError_t launch_attn(const AttnLaunch &a, const AttnPlan &p, hipStream_t st)
{
    if (p.wide && p.out_cols == 256) launch_wide<320, 256>(a, p.wq, st);
    else if (p.wide) launch_wide<576, 512>(a, p.wq, st);
    else if (a.bf16) launch_main<true>(a, p, st);
    else launch_main<false>(a, p, st);
    const int n_join = p.wide || p.direct ? 0 : a.B * a.Hq;
    const int each = kv_weight_positions(a.Hq / a.Hkv);
    const int n_weights = a.acc_out ? a.B * a.Hkv * ((a.cap + each - 1) / each) : 0;
    if (n_join + n_weights > 0) attn_finish_kernel<<<n_join + n_weights, KV_NT, 0, st>>>(a, n_join, p.wide);
    return hipGetLastError();
}

}  // namespace coli
