// shared.hip -- attention of one new token per sequence where groups of
// sequences begin with the same pages ("Add GLM-5.3-Flash (glm5next) support
// with ROCmFP mix qtypes (105/106)", section "MLA/DSA": softmax attention over
// the cached positions).
//
// The softmax over a sequence's positions is joined from two parts: the shared
// pages, for which the query heads of all the group's sequences stand side by
// side as the heads of one sequence, so that each key and value is read once
// for all of them; and the sequence's own positions behind.  Both leave
// references m, sums l and unnormalised outputs O, as a sequence that is cut
// does, and one kernel joins them:
//   out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i
#include "attend.h"

namespace coli {

// One (sequence, query head) a workgroup.  The own parts come first, then the
// shared pages'.
template <bool WIDE>
__global__ __launch_bounds__(KV_NT) void attn_shared_join_kernel(AttnLaunch own, AttnLaunch pre)
{
    __shared__ __attribute__((aligned(16))) float red[KV_NT * 4];
    __shared__ float factor[2 * KV_MAX_WG];
    const int tid = threadIdx.x, lane = tid & 63;
    const int bq = blockIdx.x, b = bq / own.Hq, hq = bq - b * own.Hq;
    const int G = own.Hq / own.Hkv, h = hq / G, qi = hq - h * G;
    int before, total;
    kv_prefix<KV_OWN>(own, b, &before, &total);
    const KvParts p = kv_parts<KV_OWN>(own, b, h * own.q_tiles + qi / own.tile_rows, before, total);
    const int n_own = p.steps == 0 ? 0 : p.w1 - p.w0 + 1, q_own = qi % own.tile_rows;
    // (a row that is not cut is one part, in its queries' places)
    int n_pre = 0, q_pre = 0;
    KvParts pp{};
    const int pages = kv_shared(own, b);
    if (pages > 0 && kv_left(own, b) == pages) {
        int g = -1;
        for (int c = 0; g < 0 && c < pre.n_groups; c += 64) {
            const bool here = c + lane < pre.n_groups && kv_group_first(pre, c + lane) <= b && b < kv_group_end(pre, c + lane);
            const uint64_t mask = __ballot(here);
            if (mask) g = c + __ffsll((unsigned long long)mask) - 1;
        }
        if (g >= 0) {
            kv_prefix<KV_PREFIX>(pre, g, &before, &total);
            const int i = (b - kv_group_first(pre, g)) * G + qi;
            pp = kv_parts<KV_PREFIX>(pre, g, h * kv_tiles<KV_PREFIX>(pre, g) + i / pre.tile_rows, before, total);
            n_pre = pp.steps == 0 ? 0 : pp.w1 - pp.w0 + 1;
            q_pre = i % pre.tile_rows;
        }
    }
    const int n = n_own + n_pre;
    if (n == 0) return kv_write_empty(own, bq, 1);
    auto query = [&](int w) {                 // of part w, that of a cut row: row of part_ml
        return w < n_own ? (size_t)p.slot(p.w0 + w) * own.tile_rows + q_own
                         : (size_t)pp.slot(pp.w0 + w - n_own) * pre.tile_rows + q_pre;
    };
    auto whole = [&](int w) { return w < n_own ? n_own == 1 : n_pre == 1; };
    auto ml = [&](int w) {
        return whole(w) ? (w < n_own ? own.full_ml : pre.full_ml) + 2 * (size_t)bq
                        : (w < n_own ? own.part_ml : pre.part_ml) + 2 * query(w);
    };

    float mx = -INFINITY;
    for (int w = lane; w < n; w += 64) mx = fmaxf(mx, ml(w)[0]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
    const float ref = mx == -INFINITY ? 0.f : mx;
    float l = 0.f;
    for (int w = lane; w < n; w += 64) {
        const float f = __builtin_amdgcn_exp2f(ml(w)[0] - ref);
        l += ml(w)[1] * f;
        if (tid < 64) factor[w] = f;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) l += __shfl_xor(l, off);
    __syncthreads();

    // groups of threads take every ng-th part, 4 columns a thread
    const int cols = own.Dv / 4, ng = KV_NT / cols, grp = tid / cols, col = tid % cols;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    if (grp < ng) {
#pragma unroll 4
        for (int w = grp; w < n; w += ng) {
            const float *part = w < n_own ? (whole(w) ? own.full_o : own.part_o) : whole(w) ? pre.full_o : pre.part_o;
            const size_t q = whole(w) ? (size_t)bq : query(w);
            // (the wide kernel's parts: lanes side by side, 32 queries at a time)
            const size_t at = WIDE && !whole(w) ? (q >> 5) * 32 * own.out_cols + ((size_t)(col >> 1) * 64 + (col & 1) * 32 + (q & 31)) * 4
                                                : q * own.Dv + 4 * col;
            acc += *reinterpret_cast<const f32x4 *>(part + at) * factor[w];
        }
        *reinterpret_cast<f32x4 *>(red + 4 * tid) = acc;
    }
    __syncthreads();
    if (tid < cols) {
        for (int x = 1; x < ng; ++x) acc += *reinterpret_cast<const f32x4 *>(red + 4 * (x * cols + col));
        const float inv = kv_inverse(l);
        const size_t at = (size_t)bq * own.Dv + 4 * col;
        if (own.bf16)
            *reinterpret_cast<u32x2 *>((uint16_t *)own.out + at) =
                u32x2{pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv)};
        else *reinterpret_cast<f32x4 *>((float *)own.out + at) = acc * inv;
    }
    if (tid == 0) kv_write_lse(own, bq, mx, l);
}

SharedPlan attn_shared_plan(int B, int Hq, int Hkv, int Dk, int Dv, bool bf16, bool latent, int n_groups, int entries)
{
    SharedPlan s{};
    const int G = Hq / Hkv;
    // query heads that a group has for each cache head, by the mean
    const long queries = ((long)B * G + n_groups - 1) / (n_groups > 0 ? n_groups : 1);
    AttnPlan p = attn_plan(B, Hq, Hkv, Dk, Dv, bf16, latent, entries);
    // the lengths behind the shared pages are on the device: rows are cut
    p.wide = bf16 && (Dk > 256 || (latent && Dk > 128 && queries > KV_QT));
    p.direct = false;
    p.waves = KV_WAVES;
    const int d = Dk > Dv ? Dk : Dv;
    if (p.wide) {
        p.out_cols = (Dk <= 320 && Dv <= 256) ? 256 : 512;
        p.n_wg = KW_MAX_WG;
        p.min_units = KV_ROW_UNITS;
        s.own = s.pre = p;
        s.own.wq = G <= 32 ? 1 : G <= 64 ? 2 : 4;
        s.pre.wq = queries <= 32 ? 1 : queries <= 64 ? 2 : 4;
        s.own.tile_rows = 32 * s.own.wq;
        s.pre.tile_rows = 32 * s.pre.wq;
    } else {
        p.tile_rows = KV_QT;
        p.out_cols = Dv;
        p.tier = d <= 64 ? 64 : d <= 128 ? 128 : d <= 192 && !bf16 ? 192 : d <= 256 ? 256 : (d <= 320 && Dv <= 256) ? 320 : 512;
        p.n_wg = 256 * (d <= (bf16 ? 128 : 64) ? 2 : 1);
        p.min_units = 4;
        s.own = s.pre = p;
    }
    s.own.q_tiles = (G + s.own.tile_rows - 1) / s.own.tile_rows;
    s.pre.q_tiles = 0;                        // each group's own
    return s;
}

template <bool BF16, KvPart PART>
static void launch_tiles(const AttnLaunch &a, const AttnPlan &p, hipStream_t st)
{
    if (p.tier == 64) attn_kernel<BF16, 64, 64, KV_WAVES, PART><<<a.n_wg, KV_NT, 0, st>>>(a);
    else if (p.tier == 128) attn_kernel<BF16, 128, 128, KV_WAVES, PART><<<a.n_wg, KV_NT, 0, st>>>(a);
    else if (p.tier == 256) attn_kernel<BF16, 256, 256, KV_WAVES, PART><<<a.n_wg, KV_NT, 0, st>>>(a);
    else if constexpr (!BF16) {
        if (p.tier == 192) attn_kernel<BF16, 192, 192, KV_WAVES, PART><<<a.n_wg, KV_NT, 0, st>>>(a);
        else if (p.tier == 320) attn_kernel<BF16, 320, 256, KV_WAVES, PART><<<a.n_wg, KV_NT, 0, st>>>(a);
        else attn_kernel<BF16, 576, 512, KV_WAVES, PART><<<a.n_wg, KV_NT, 0, st>>>(a);
    }
}

template <int DK, int DV, int WQ, KvPart PART>
static void launch_wide(const AttnLaunch &a, hipStream_t st)
{
    if (a.Dk == DK) attn_wide_kernel<DK, DV, WQ, KW_NONE, PART><<<a.n_wg, KV_NT, 0, st>>>(a);
    else if (a.Dk >= DV) attn_wide_kernel<DK, DV, WQ, KW_TAIL, PART><<<a.n_wg, KV_NT, 0, st>>>(a);
    else attn_wide_kernel<DK, DV, WQ, KW_BOTH, PART><<<a.n_wg, KV_NT, 0, st>>>(a);
}

template <int DK, int DV, KvPart PART>
static void launch_wide(const AttnLaunch &a, int wq, hipStream_t st)
{
    if (wq == 1) launch_wide<DK, DV, 1, PART>(a, st);
    else if (wq == 2) launch_wide<DK, DV, 2, PART>(a, st);
    else launch_wide<DK, DV, 4, PART>(a, st);
}

template <KvPart PART>
static void launch_part(const AttnLaunch &a, const AttnPlan &p, hipStream_t st)
{
    if (p.wide && p.out_cols == 256) launch_wide<320, 256, PART>(a, p.wq, st);
    else if (p.wide) launch_wide<576, 512, PART>(a, p.wq, st);
    else if (a.bf16) launch_tiles<true, PART>(a, p, st);
    else launch_tiles<false, PART>(a, p, st);
}

hipError_t launch_attn_shared(const AttnLaunch &own, const AttnLaunch &pre, const SharedPlan &p, hipStream_t st)
{
    launch_part<KV_OWN>(own, p.own, st);
    launch_part<KV_PREFIX>(pre, p.pre, st);
    if (p.own.wide) attn_shared_join_kernel<true><<<own.B * own.Hq, KV_NT, 0, st>>>(own, pre);
    else attn_shared_join_kernel<false><<<own.B * own.Hq, KV_NT, 0, st>>>(own, pre);
    return hipGetLastError();
}

}  // namespace coli
