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
#include "device_common.h"
#include "kernels.h"

namespace coli {

constexpr int KV_NT = 256;                    // threads per workgroup (4 waves)
constexpr int KV_WAVES = KV_NT / 64;
constexpr int KV_STEP = 32;                   // positions per step of a wave
constexpr int KV_QT = 16;                     // query heads per matrix tile

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short bf16x8s __attribute__((ext_vector_type(8)));

// Steps of sequence b (per cache head and query tile).
__device__ __forceinline__ int kv_len(const AttnLaunch &a, int b)
{
    return a.idx ? a.idx_k : min(max(a.lens[b], 0), a.cap);
}
__device__ __forceinline__ int kv_steps(int n) { return (n + KV_STEP - 1) / KV_STEP; }

__device__ __forceinline__ int block_sum(int v, int32_t *red)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
    __syncthreads();
    if (lane == 0) red[wave] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < KV_WAVES; ++w) s += red[w];
    return s;
}

// Steps of all sequences before b, and of all sequences (per unit of
// Hkv * query tiles).
__device__ __forceinline__ void kv_prefix(const AttnLaunch &a, int b, int32_t *red, int *before, int *total)
{
    int lo = 0, all = 0;
    for (int i = threadIdx.x; i < a.B; i += KV_NT) {
        const int st = kv_steps(kv_len(a, i));
        all += st;
        lo += (i < b) ? st : 0;
    }
    *before = block_sum(lo, red);
    *total = block_sum(all, red);
}

// Units (steps) of one workgroup's range.
__device__ __forceinline__ int kv_range(const AttnLaunch &a, int units)
{
    return max((units + a.n_wg - 1) / a.n_wg, a.min_units);
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

template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(KV_NT) void attn_kernel(AttnLaunch a)
{
    using KT = KvTile<BF16, DK, DV>;
    using T = typename KT::T;
    constexpr int EPL = KT::EPL, KC = KT::KC, VE = KT::VE, VC = KT::VC, VW = KT::VW;
    constexpr int RS = DV + 4;                // padded row of the join buffer
    __shared__ __attribute__((aligned(16))) float red[2][KV_QT][RS];
    __shared__ float red_m[KV_WAVES][KV_QT], red_l[KV_WAVES][KV_QT];
    __shared__ int32_t scan[KV_WAVES];
    __shared__ int32_t found[2];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int j = lane & 15, g = lane >> 4;
    const int G = a.Hq / a.Hkv;
    const int R = a.Hkv * a.q_tiles;

    // ---- this workgroup's range and its first sequence ----
    int total;
    {
        int sum = 0;
        for (int i = tid; i < a.B; i += KV_NT) sum += kv_steps(kv_len(a, i));
        total = block_sum(sum, scan) * R;
    }
    const int range = kv_range(a, total);
    int u = blockIdx.x * range;               // at most n_wg * range: below 2^31 by the host's check
    if (u >= total) return;
    const int u_end = min(u + range, total);
    {
        int base = 0;
        if (tid == 0) found[0] = -1;
        for (int c = 0; c < a.B; c += KV_NT) {
            const int st = (c + tid < a.B) ? kv_steps(kv_len(a, c + tid)) : 0;
            __syncthreads();
            const int incl = block_scan_incl<KV_WAVES>(st, scan) + base;
            if (u >= (incl - st) * R && u < incl * R) {
                found[0] = c + tid;
                found[1] = (incl - st) * R;
            }
            __syncthreads();
            base += scan[KV_WAVES - 1];
            if (found[0] >= 0) break;
        }
    }
    int b = found[0];
    int n = kv_len(a, b), steps = kv_steps(n);
    int row = (u - found[1]) / steps, s0 = (u - found[1]) % steps;
    const int u_begin = u;

    const T *kpool = (const T *)a.k;
    const T *vpool = (const T *)(a.v ? a.v : a.k);
    const int vstride = a.v ? a.Dv : a.Dk;

    while (u < u_end) {
        const int s1 = min(steps, s0 + (u_end - u));
        const int h = row / a.q_tiles, q0 = (row % a.q_tiles) * KV_QT;
        const int nq = min(KV_QT, G - q0);    // query heads of this tile
        const size_t qrow = (size_t)b * a.Hq + h * G + q0;
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
        auto rows_of = [&](int s) {
            int p = s * KV_STEP + (lane & 31);
            bool ok = p < n && s < s1;
            if (a.idx) {
                p = ok ? a.idx[(size_t)b * a.idx_k + p] : -1;
                ok = p >= 0 && p < len;
            }
            int r = -1;
            if (ok) {
                const int pg = a.table[(size_t)b * a.max_pages + (p >> a.page_shift)];
                if (pg >= 0 && pg < a.n_pages)
                    r = (int)((((uint32_t)pg * (uint32_t)a.Hkv + (uint32_t)h) << a.page_shift) +
                              (uint32_t)(p & ((1 << a.page_shift) - 1)));
            }
            return r;
        };
        u32x4 kf[2][KC];
        auto load_keys = [&](int rows) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int r = max(__shfl(rows, 16 * t + j), 0);
                const T *p = kpool + (size_t)r * a.Dk;
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const int d = (4 * c + g) * EPL;      // past the key's width: a zero of the query meets it
                    kf[t][c] = *reinterpret_cast<const u32x4 *>(p + (d < a.Dk ? d : 0));
                }
            }
        };
        uint32_t vf[VC][8][VW];
        auto load_values = [&](int rows) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = max(__shfl(rows, 16 * (i >> 2) + 4 * g + (i & 3)), 0);
                const T *p = vpool + (size_t)r * vstride;
#pragma unroll
                for (int c = 0; c < VC; ++c) {
                    const int d = (16 * c + j) * VE;      // past the value's width: columns that are not written
                    const T *src = p + (d < a.Dv ? d : 0);
                    if constexpr (VW == 4) {
                        const u32x4 x = *reinterpret_cast<const u32x4 *>(src);
#pragma unroll
                        for (int w = 0; w < 4; ++w) vf[c][i][w] = x[w];
                    } else {
                        const u32x2 x = *reinterpret_cast<const u32x2 *>(src);
                        vf[c][i][0] = x[0];
                        vf[c][i][1] = x[1];
                    }
                }
            }
        };

        int s = s0 + wave;
        int rows = rows_of(s), rows_next = rows_of(s + KV_WAVES);
        if (s < s1) {
            load_keys(rows);
            load_values(rows);
        }
        for (; s < s1; s += KV_WAVES) {
            const bool more = s + KV_WAVES < s1;
            // ---- scores: D[key][query] = K Q^T, two tiles of 16 keys ----
            f32x4 sc[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                sc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    if constexpr (BF16) {
                        sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(kf[t][c]), as_bf16(qf[c]), sc[t], 0, 0, 0);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(kf[t][c][e]),
                                                                        __uint_as_float(qf[c][e]), sc[t], 0, 0, 0);
                    }
                }
            }
            const int rows_now = rows;
            rows = rows_next;
            if (more) load_keys(rows);
            rows_next = rows_of(s + 2 * KV_WAVES);

            // ---- weights: lane (j, g) holds query j, positions 16 t + 4 g + r ----
            float t2[8];
            const uint64_t hidden = __ballot(rows_now < 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) t2[i] = fmaf(sc[i >> 2][i & 3], a.scale_hi, sc[i >> 2][i & 3] * a.scale_lo);
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
            if (hidden) {                     // what stands in hidden rows (NaN, infinities) must not count
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (__shfl(rows_now, 16 * (i >> 2) + 4 * g + (i & 3)) < 0) {
#pragma unroll
                        for (int c = 0; c < VC; ++c)
#pragma unroll
                            for (int x = 0; x < VW; ++x) vf[c][i][x] = 0u;
                    }
            }
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
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int c = 0; c < VC; ++c)
#pragma unroll
                        for (int e = 0; e < VE; ++e)
                            o[c][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(vf[c][i][e]), w[i], o[c][e],
                                                                          0, 0, 0);
            }
            if (more) load_values(rows);
        }

        // ---- the four waves' parts become one ----
        l = quad_sum(l);
        if (g == 0) {
            red_m[wave][j] = m;
            red_l[wave][j] = l;
        }
        __syncthreads();
        float ma = red_m[0][j];
#pragma unroll
        for (int w = 1; w < KV_WAVES; ++w) ma = fmaxf(ma, red_m[w][j]);
        const float f = (m == -INFINITY) ? 0.f : __builtin_amdgcn_exp2f(m - ma);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if ((wave >> 1) == half && j < nq) {
#pragma unroll
                for (int c = 0; c < VC; ++c)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float *dst = &red[wave & 1][j][(16 * c + 4 * g + r) * VE];
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            const float v = o[c][e][r] * f;
                            dst[e] = half ? dst[e] + v : v;
                        }
                    }
            }
            __syncthreads();
        }
        const bool whole = s0 == 0 && s1 == steps;
        const int slot = 2 * blockIdx.x + (u == u_begin ? 0 : 1);
        for (int i = tid; i < nq * DV; i += KV_NT) {
            const int q = i / DV, d = i % DV;
            if (d >= a.Dv) continue;
            const float v = red[0][q][d] + red[1][q][d];
            float mq = red_m[0][q], lq = 0.f;
#pragma unroll
            for (int w = 1; w < KV_WAVES; ++w) mq = fmaxf(mq, red_m[w][q]);
#pragma unroll
            for (int w = 0; w < KV_WAVES; ++w)
                lq += (red_m[w][q] == -INFINITY) ? 0.f : red_l[w][q] * __builtin_amdgcn_exp2f(red_m[w][q] - mq);
            if (whole) {
                const float y = lq > 0.f ? v / lq : 0.f;
                if constexpr (BF16) ((uint16_t *)a.out)[(qrow + q) * a.Dv + d] = f32_to_bf16_bits(y);
                else ((float *)a.out)[(qrow + q) * a.Dv + d] = y;
                if (d == 0) {
                    if (a.lse) a.lse[qrow + q] = lq > 0.f ? (mq + log2f(lq)) * 0.6931471805599453f : -INFINITY;
                    if (a.stats) {
                        a.stats[2 * (qrow + q)] = mq == -INFINITY ? 0.f : mq;
                        a.stats[2 * (qrow + q) + 1] = lq > 0.f ? 1.f / lq : 0.f;
                    }
                }
            } else {
                a.part_o[((size_t)slot * KV_QT + q) * a.Dv + d] = v;
                if (d == 0) {
                    a.part_ml[((size_t)slot * KV_QT + q) * 2] = mq;
                    a.part_ml[((size_t)slot * KV_QT + q) * 2 + 1] = lq;
                }
            }
        }
        __syncthreads();                      // the join buffer is free again

        u += s1 - s0;
        s0 = 0;
        if (++row == R) {
            row = 0;
            do {
                ++b;
                n = b < a.B ? kv_len(a, b) : 1;
                steps = kv_steps(n);
            } while (steps == 0);
        }
    }
}

// One workgroup per (sequence, query head): joins the parts that the ranges'
// borders left of it, or writes an empty sequence's zeros.  The parts are
// summed in the order of the positions.
__global__ __launch_bounds__(KV_NT) void attn_join_kernel(AttnLaunch a)
{
    __shared__ int32_t scan[KV_WAVES];
    __shared__ __attribute__((aligned(16))) float red[KV_NT * 4];
    const int tid = threadIdx.x;
    const int b = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq;
    const int G = a.Hq / a.Hkv, R = a.Hkv * a.q_tiles;
    int before, total;
    kv_prefix(a, b, scan, &before, &total);
    const int steps = kv_steps(kv_len(a, b));
    const int qi = hq % G, row = hq / G * a.q_tiles + qi / KV_QT, q = qi % KV_QT;
    if (steps == 0) {
        for (int d = tid; d < a.Dv; d += KV_NT) {
            if (a.bf16) ((uint16_t *)a.out)[(size_t)blockIdx.x * a.Dv + d] = 0;
            else ((float *)a.out)[(size_t)blockIdx.x * a.Dv + d] = 0.f;
        }
        if (tid == 0) {
            if (a.lse) a.lse[blockIdx.x] = -INFINITY;
            if (a.stats) a.stats[2 * blockIdx.x] = a.stats[2 * blockIdx.x + 1] = 0.f;
        }
        return;
    }
    const int range = kv_range(a, total * R);
    const int u0 = before * R + row * steps, u1 = u0 + steps;
    const int w0 = u0 / range, w1 = (u1 - 1) / range;
    if (w0 == w1) return;                     // one range holds all of it
    const int first_slot = 2 * w0 + (u0 == w0 * range ? 0 : 1);
    auto slot_of = [&](int w) { return (size_t)(w == w0 ? first_slot : 2 * w) * KV_QT + q; };

    float mx = -INFINITY;
    for (int w = w0 + (tid & 63); w <= w1; w += 64) mx = fmaxf(mx, a.part_ml[slot_of(w) * 2]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
    const float ref = mx == -INFINITY ? 0.f : mx;
    float l = 0.f;
    for (int w = w0 + (tid & 63); w <= w1; w += 64)
        l += a.part_ml[slot_of(w) * 2 + 1] * __builtin_amdgcn_exp2f(a.part_ml[slot_of(w) * 2] - ref);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) l += __shfl_xor(l, off);

    // groups of threads take every ng-th part, 4 columns a thread
    const int cols = a.Dv / 4, ng = KV_NT / cols, grp = tid / cols, col = tid % cols;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    if (grp < ng) {
        for (int w = w0 + grp; w <= w1; w += ng) {
            const size_t sl = slot_of(w);
            acc += *reinterpret_cast<const f32x4 *>(a.part_o + sl * a.Dv + 4 * col) *
                   __builtin_amdgcn_exp2f(a.part_ml[sl * 2] - ref);
        }
        *reinterpret_cast<f32x4 *>(red + 4 * tid) = acc;
    }
    __syncthreads();
    if (tid < cols) {
        for (int x = 1; x < ng; ++x) acc += *reinterpret_cast<const f32x4 *>(red + 4 * (x * cols + col));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float y = l > 0.f ? acc[x] / l : 0.f;
            const size_t at = (size_t)blockIdx.x * a.Dv + 4 * col + x;
            if (a.bf16) ((uint16_t *)a.out)[at] = f32_to_bf16_bits(y);
            else ((float *)a.out)[at] = y;
        }
    }
    if (tid == 0) {
        if (a.lse) a.lse[blockIdx.x] = l > 0.f ? (ref + log2f(l)) * 0.6931471805599453f : -INFINITY;
        if (a.stats) {
            a.stats[2 * blockIdx.x] = ref;
            a.stats[2 * blockIdx.x + 1] = l > 0.f ? 1.f / l : 0.f;
        }
    }
}

// Running weights: acc_out = acc_in + sum over the cache head's query heads
// of e^(t - m) / l, four positions a thread.
__global__ __launch_bounds__(KV_NT) void attn_weights_kernel(AttnLaunch a)
{
    const int chunks = (a.cap + 4 * KV_NT - 1) / (4 * KV_NT);
    const int bh = blockIdx.x / chunks, b = bh / a.Hkv, h = bh % a.Hkv, G = a.Hq / a.Hkv;
    const int n = min(max(a.lens[b], 0), a.cap);
    const int p = ((int)blockIdx.x % chunks * KV_NT + (int)threadIdx.x) * 4;
    if (p >= n) return;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < G; ++i) {
        const size_t qrow = (size_t)b * a.Hq + h * G + i;
        const f32x4 t = *reinterpret_cast<const f32x4 *>(a.scores + qrow * a.s_ld + p);
        const float m = a.stats[2 * qrow], inv = a.stats[2 * qrow + 1];
#pragma unroll
        for (int x = 0; x < 4; ++x) sum[x] += __builtin_amdgcn_exp2f(t[x] - m) * inv;
    }
    const size_t at = (size_t)bh * a.ld + p;
    if (p + 4 <= n) {
        if (a.acc_in) sum += *reinterpret_cast<const f32x4 *>(a.acc_in + at);
        *reinterpret_cast<f32x4 *>(a.acc_out + at) = sum;
    } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (p + x < n) a.acc_out[at + x] = sum[x] + (a.acc_in ? a.acc_in[at + x] : 0.f);
    }
}

// Workgroups of the main kernel: its ranges.
int attn_workgroups() { return 1024; }
int attn_q_tiles(int Hq, int Hkv) { return (Hq / Hkv + KV_QT - 1) / KV_QT; }
int attn_tile_rows() { return KV_QT; }

template <bool BF16>
static void launch_main(const AttnLaunch &a, hipStream_t st)
{
    const int d = max(a.Dk, a.Dv);
    if (d <= 64) attn_kernel<BF16, 64, 64><<<a.n_wg, KV_NT, 0, st>>>(a);
    else if (d <= 128) attn_kernel<BF16, 128, 128><<<a.n_wg, KV_NT, 0, st>>>(a);
    else if (d <= 256) attn_kernel<BF16, 256, 256><<<a.n_wg, KV_NT, 0, st>>>(a);
    else attn_kernel<BF16, 576, 512><<<a.n_wg, KV_NT, 0, st>>>(a);
}

hipError_t launch_attn(const AttnLaunch &a, hipStream_t st)
{
    if (a.bf16) launch_main<true>(a, st);
    else launch_main<false>(a, st);
    attn_join_kernel<<<a.B * a.Hq, KV_NT, 0, st>>>(a);
    if (a.acc_out) {
        const int chunks = (a.cap + 4 * KV_NT - 1) / (4 * KV_NT);
        attn_weights_kernel<<<a.B * a.Hkv * chunks, KV_NT, 0, st>>>(a);
    }
    return hipGetLastError();
}

}  // namespace coli
