// attend.hip -- what follows the attention kernels of attend.h (joins, running
// weights), how a call is cut, and its launches.
#include "attend.h"

namespace coli {

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
