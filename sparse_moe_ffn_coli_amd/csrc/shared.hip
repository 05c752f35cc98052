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

// ---- shared pages of many query heads ------------------------------------------
// With 64 sequences of four query heads a cache head meets 256 queries: 128
// products a byte of the cache, so the matrix cores bind and not HBM.  Each
// key and value is brought into LDS once per workgroup (copies that pass no
// registers, a ring of 32-position stages), every wave takes 32 queries on
// 32 x 32 x 16 matrix tiles, as the wide latent kernel does:
//   scores  D[key][query] = K Q^T
//   output  O^T[column][query] += V^T w   (values by the transposing LDS read)
// Eight waves (four where rows are 256 wide: twice the registers), two a SIMD:
// one's softmax runs while the other multiplies.  WQ of them have different
// queries; the waves of a query tile split the positions, NW / WQ stages a
// round, and are joined in LDS at the end of a row.
// LDS rows are RK or RV chunks of 16 bytes (a power of two), chunk c of row r
// at c XOR kp_swz(r): 16 rows of one chunk (scores) and 4 rows of 4 chunks
// (output) fall in distinct banks.
// 64 sequences of 4 heads a cache head behind 32768 positions, 8 cache heads of
// 128: 62 us, 52 GFLOP with the weights' second parts (0.84 PFLOP/s; the
// library's large product reaches 1.32).  A round of 1536 cycles of products
// takes some 3000: a weight's multiply, exponential, sum and two roundings are
// 16 to 20 issue cycles, of two waves a SIMD.  At 192 / 128 elements 29 to 35
// registers spill (24 sequences behind 32768 positions 78 us a call, 256 / 256
// 107; 192 / 192 runs as 256, 101).
constexpr int KP_BLOCK = 32;                  // stages whose rows are looked up at a time

template <int R>
__device__ __forceinline__ int kp_swz(int row)
{
    if constexpr (R == 8) return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);      // two rows to a bank round
    else return kw_swz(row);
}
constexpr int kp_chunks(int width) { return width <= 64 ? 8 : width <= 128 ? 16 : 32; }

// 2^(scale (score - ref)): the reference is a score, and what is scaled is how
// far the others are from it.  So the factor's rounding (one float) counts for
// the distance only, equal scores have equal weights however large they are, and
// only the reference itself needs the factor's two parts (kv_scaled).  (A
// distance past fp32's end has no weight: a scale that gave it one would be
// below 1e-36.)
__device__ __forceinline__ float kp_weight(float score, float scale, float ref)
{
    return __builtin_amdgcn_exp2f((score - ref) * scale);
}

// Two fp32 to bf16 in one instruction (pack_bf16 takes four).
__device__ __forceinline__ uint32_t kp_pack(float lo, float hi)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

struct KpGroup {
    int first, queries, tiles;                // first sequence, query heads of a cache head, their tiles
};
__device__ __forceinline__ KpGroup kp_group(const AttnLaunch &a, int b)
{
    KpGroup g;
    g.first = kv_group_first(a, b);
    g.queries = (kv_group_end(a, b) - g.first) * (a.Hq / a.Hkv);
    g.tiles = (g.queries + a.tile_rows - 1) / a.tile_rows;
    return g;
}
template <int DK, int DV, int WQ, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(NW / 4, NW / 4))) void attn_prefix_kernel(AttnLaunch a)
{
    constexpr int WK = NW / WQ;
    constexpr int RK = kp_chunks(DK), RV = kp_chunks(DV);
    constexpr int KB = KW_ROWS * RK * 16, STAGE = KB + KW_ROWS * RV * 16;         // bytes of a stage's keys, and of all
    constexpr int CK = RK / 2, CPS = CK + RV / 2;             // copy instructions of a stage
    constexpr int OUT = 32 * DV;                              // floats of a query tile's output
    constexpr int RING = 147456 / STAGE < 8 ? 147456 / STAGE : 8;                 // stages in LDS; a row's outputs fit too
    // A round is a stage for each of the WK position groups, a barrier every PB
    // rounds.  A round's output products follow in the next round, between its
    // weights, so that the matrix cores run during the softmax.  (Half of the
    // waves a phase later than the others, 64 sequences of 4 heads behind 32768
    // positions: 64.0 us, 63.1 without.)
    constexpr int PB = RING / WK >= 6 ? 2 : 1, BLOCKS = RING / (WK * PB);         // barriers' spans in the ring
    constexpr int AHEAD = BLOCKS - 2;                         // spans in flight beside the one computed and the one before
    constexpr int CPW = CPS * WK * PB / NW;                   // copies of a wave in a span
    constexpr int KS = DK / 16, DT = DV / 32;
    static_assert(CPS * WK * PB % NW == 0 && AHEAD >= 1 && (AHEAD - 1) * CPW < 64, "copies of a round");
    static_assert(NW * OUT * 4 <= RING * STAGE, "outputs of all waves");
    __shared__ __attribute__((aligned(256))) char ring[RING * STAGE];
    __shared__ int32_t rows_s[2][KP_BLOCK * KW_ROWS];         // pool rows of the stages' positions, -1: hidden
    __shared__ float red_m[NW][32], red_l[NW][32];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int qt = wave % WQ, kb = wave / WQ;
    const int ql = lane & 31, hi = lane >> 5;
    KvRange rg;
    if (!kv_first<KV_PREFIX>(a, 1, rg)) return;
    KpGroup grp = kp_group(a, rg.b);
    int u = rg.u, b = rg.b, n = rg.n, steps = rg.steps, row = rg.row, s0 = rg.s0;
    const int u_begin = u, u_end = rg.u_end;
    const uint32_t ring_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)ring;
    const uint64_t kpool = (uint64_t)a.k, vpool = (uint64_t)(a.v ? a.v : a.k);
    // The queries take scale's sign, so that the largest product is the largest
    // score.
    // A scale of zero becomes zero queries (of which an infinity is no number, as its product with the scale): the
    // scores of hidden positions are infinities.
    const bool zero = a.scale_size == 0.f;
    const float scale = zero ? 1.f : a.scale_size;
    const uint32_t flip = a.scale_hi < 0.f ? 0x80008000u : 0u;
    const uint32_t k_bytes = a.Dk * 2, v_bytes = a.v ? a.Dv * 2 : k_bytes;        // from a row to the next

    // this lane's places in a stage: key row ql, chunk hi; and the transposing reads' rows 4 hi + rr, of whose columns
    // bit 4 of the lane gives the sixteen
    const int key_at = ql * (RK * 16) + ((hi ^ kp_swz<RK>(ql)) << 4);
    const int rr = (lane & 15) >> 2;
    const int val_at = KB + (4 * hi + rr) * (RV * 16) +
                       (((2 * ((lane >> 4) & 1) + ((lane >> 1) & 1)) ^ kp_swz<RV>(4 * hi + rr)) << 4) + (lane & 1) * 8;

    auto advance = [&] {
        u += kv_units(n) - s0;
        s0 = 0;
        const int was = b;
        kv_next_row<KV_PREFIX>(a, 1, b, n, steps, row);
        if (b != was && u < u_end) grp = kp_group(a, b);
    };
    for (;; advance()) {
        if (u >= u_end) return;
        const int s1 = min(steps, s0 + (u_end - u));
        if (s0 >= steps) continue;            // a row's units past its steps
        const int first = grp.first, h = row / grp.tiles, tq0 = (row - h * grp.tiles) * (32 * WQ), q0 = tq0 + 32 * qt;
        const int nq = grp.queries - q0;      // query heads of this wave's tile (may be none)
        const int seg = s1 - s0, rounds = (seg + 2 * WK - 1) / (2 * WK) * 2;     // (pairs: a stage past the end is hidden)

        u32x4 qr[KS];
        {
            const uint16_t *q = (const uint16_t *)a.q + kv_query_row(a, first, h, q0 + min(ql, max(nq, 1) - 1)) * a.Dk;
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                const int d = 16 * c + 8 * hi;
                qr[c] = u32x4{0u, 0u, 0u, 0u};
                if (ql < nq && d < a.Dk) qr[c] = *reinterpret_cast<const u32x4 *>(q + d);
            }
        }
        // pool rows of the block of stages that holds stage t0 (a multiple of KP_BLOCK)
        auto look_up = [&](int t0) {
            constexpr int PER = KP_BLOCK * KW_ROWS / (64 * NW);
            const int end = min(n, s1 * KV_STEP);
            int p[PER], pg[PER];
#pragma unroll
            for (int x = 0; x < PER; ++x) {
                p[x] = (s0 + t0) * KV_STEP + tid + x * (64 * NW);
                pg[x] = a.table[(size_t)first * a.max_pages + (min(p[x], end - 1) >> a.page_shift)];
            }
#pragma unroll
            for (int x = 0; x < PER; ++x)
                rows_s[(t0 / KP_BLOCK) & 1][tid + x * (64 * NW)] =
                    p[x] < end && pg[x] >= 0 && pg[x] < a.n_pages ? kv_pool_row(a, pg[x], h, p[x]) : -1;
        };
        // The wave's copies of span r: copy x of a wave is number NW x + wave of the span's.  Their addresses are formed
        // a span ahead.
        uint64_t from[CPW];
        auto address = [&](int r) {
#pragma unroll
            for (int x = 0; x < CPW; ++x) {
                const int t = r * (WK * PB) + NW * x / CPS, i = NW * x % CPS + wave;
                const int32_t *rows = rows_s[(t / KP_BLOCK) & 1] + (t % KP_BLOCK) * KW_ROWS;
                auto part = [&](auto chunks, int i, uint64_t pool, uint32_t bytes, uint32_t width) {
                    constexpr int R = decltype(chunks)::value;
                    const int at = i * (64 / R) + lane / R;
                    const uint32_t off = ((lane % R) ^ kp_swz<R>(at)) << 4;
                    const int row = rows[at];
                    from[x] = row >= 0 && off < width ? pool + (uint64_t)(uint32_t)row * bytes + off : (uint64_t)kv_zeros;
                };
                if (CK % NW == 0 ? NW * x % CPS < CK : i < CK) part(KwInt<RK>{}, i, kpool, k_bytes, k_bytes);
                else part(KwInt<RV>{}, i - CK, vpool, v_bytes, a.Dv * 2);
            }
        };
        auto issue = [&](int r) {
#pragma unroll
            for (int x = 0; x < CPW; ++x) {
                const int t = r * (WK * PB) + NW * x / CPS, i = NW * x % CPS + wave;     // (keys first, values behind them)
                kw_copy(from[x], ring_at + (t % RING) * STAGE + i * 1024);
            }
        };

        f32x16 o[DT];
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[t][i] = 0.f;
        float m = -INFINITY, l = 0.f;
        look_up(0);
        kw_barrier();
#pragma unroll 1
        for (int r = 0; r < AHEAD; ++r) {
            address(r);
            issue(r);
        }
        address(AHEAD);
        // Begin of span r: its copies have landed, the wave's and then everyone's, and all are done with the slots that
        // the copies of a later span, which go out now, are to fill.
        auto begin = [&](int r) {
            kw_wait_copies<(AHEAD - 1) * CPW>();
            kw_barrier();
            const int ahead = r + AHEAD;
            if (ahead * (WK * PB) % KP_BLOCK == 0) {
                look_up(ahead * (WK * PB));
                kw_barrier();
                address(ahead);
            }
            issue(ahead);
            address(ahead + 1);               // (at a block's end: of rows that are not looked up yet, formed again then)
        };
        bf16x8 qf[KS];
#pragma unroll
        for (int c = 0; c < KS; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                qr[c][i] ^= flip;
                if (zero) {
                    const uint32_t lo = (qr[c][i] & 0x7f80u) == 0x7f80u ? 0x7fc0u : 0u;
                    qr[c][i] = lo | ((qr[c][i] & 0x7f800000u) == 0x7f800000u ? 0x7fc00000u : 0u);
                }
            }
            qf[c] = as_bf16(qr[c]);
        }
        // Scores and their maximum; the reference, and by what the output is to be multiplied where it has moved (only where
        // a score passes it by 2^8: weights stay below 256 and the sums far inside fp32).
        f32x16 sc;
        float ref = 0.f, moved = 1.f;
        s16x4 vf[2][2][2][2];
        // Values of column tiles 2 x and 2 x + 1, read number y of eight.  Slots 0-3 of a lane are positions 16 ks + 4 hi
        // + 0..3, slots 4-7 the ones 8 further (the swizzle's second bit); a column tile is four chunks.
        auto column = [&](const char *st, int x, int y) {
            const int odd = y & 1, half = (y >> 1) & 1, ks = y >> 2, tile = 2 * x + odd;
            const int at = (val_at ^ (32 * half) ^ (64 * (tile & 3))) + (tile >> 2) * 256 + (16 * ks + 8 * half) * (RV * 16);
            vf[x & 1][odd][ks][half] =
                __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(st + at));
        };
        auto scores = [&](int t, const char *st, const char *prev, auto second) {     // second: there is a round before
            // eight fragments in a ring, the order is fixed (left to itself the compiler reads each fragment just before
            // its product)
            constexpr int KF = KS < 8 ? KS : 8;
            bf16x8 kf[KF];
            auto frag = [&](int c) { return *reinterpret_cast<const bf16x8 *>(st + (key_at ^ (32 * (c & 7))) + (c >> 3) * 256); };
            const int mine = rows_s[(t / KP_BLOCK) & 1][(t % KP_BLOCK) * KW_ROWS + ql];
#pragma unroll
            for (int c = 0; c < KF; ++c) kf[c] = frag(c);
            if constexpr (decltype(second)::value) {
#pragma unroll
                for (int y = 0; y < 8; ++y) column(prev, 0, y);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[i] = 0.f;
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[c % KF], qf[c], sc, 0, 0, 0);
                if (c + KF < KS) kf[c % KF] = frag(c + KF);
                __builtin_amdgcn_sched_barrier(0);
            }
            const uint32_t hid = (uint32_t)__ballot(mine < 0) >> (4 * hi);
            if (__ballot(hid != 0)) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (hid >> (8 * (i >> 2) + (i & 3)) & 1) sc[i] = -INFINITY;
            }
            float mx = sc[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) mx = fmaxf(mx, sc[i]);
            moved = 1.f;
            if (__ballot((mx - m) * scale > 8.f)) {
                const float mn = fmaxf(m, fmaxf(mx, __shfl_xor(mx, 32)));
                moved = (mn == -INFINITY) ? 1.f : kp_weight(m, scale, mn);
                m = mn;
                l *= moved;
            }
            ref = (m == -INFINITY) ? 0.f : m;
        };
        // Weight i (query ql, position 8 (i >> 2) + 4 hi + (i & 3)) as two bf16 parts: 16 bits of it enter the products.
        u32x4 parts[2][2][2];                 // of two rounds: high and low parts of 8 positions each
        float even;
        auto weight = [&](int i, auto to) {
            const float w = kp_weight(sc[i], scale, ref);
            l += w;
            if (i % 2 == 0) {
                even = w;
                return;
            }
            uint32_t hi2 = kp_pack(even, w);
            uint32_t lo2 = kp_pack(even - __uint_as_float(hi2 << 16), w - __uint_as_float(hi2 & 0xffff0000u));
            // (pinned: the compiler would move all of it behind the products, to where it is used)
            asm volatile("" : "+v"(hi2), "+v"(lo2), "+v"(l));
            parts[decltype(to)::value][0][i / 8][i / 2 % 4] = hi2;
            parts[decltype(to)::value][1][i / 8][i / 2 % 4] = lo2;
        };
        // Output products of one round's weights, two column tiles at a time and read one pair ahead; a weight of the next
        // round between them.
        auto output = [&](const char *st, auto of, auto with) {
            constexpr int N = 4 * DT, W = decltype(of)::value;
#pragma unroll
            for (int x = 0; x < DT / 2; ++x) {
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const int odd = y & 1, ks = y >> 2;
                    const bf16x8 vb = __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(
                        vf[x & 1][odd][ks][0], vf[x & 1][odd][ks][1], 0, 1, 2, 3, 4, 5, 6, 7));
                    o[2 * x + odd] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vb, as_bf16(parts[W][(y >> 1) & 1][ks]),
                                                                            o[2 * x + odd], 0, 0, 0);
                    if (x + 1 < DT / 2) column(st, x + 1, y);
                    if constexpr (decltype(with)::value) {
#pragma unroll
                        for (int i = (8 * x + y) * 16 / N; i < (8 * x + y + 1) * 16 / N; ++i) weight(i, KwInt<1 - W>{});
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        };
        const char *prev;
        // Round r, whose weights go to `to`; `second`: there is a round before, whose output products are due.
        auto round = [&](int r, auto to, auto second) {
            constexpr int W = decltype(to)::value;            // (r's parity)
            if (PB == 1 || W == 0) begin(r / PB);
            const int t = r * WK + kb;
            const char *st = ring + (t % RING) * STAGE;
            scores(t, st, prev, second);
            if constexpr (decltype(second)::value) {
                __builtin_amdgcn_s_setprio(1);                // (before the other wave's scores: 63.1 -> 61.2 us)
                output(prev, KwInt<1 - W>{}, KwInt<1>{});
                __builtin_amdgcn_s_setprio(0);
                if (__ballot(moved != 1.f)) {
#pragma unroll
                    for (int x = 0; x < DT; ++x) o[x] *= moved;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) weight(i, to);
            }
            prev = st;
        };
        round(0, KwInt<0>{}, KwInt<0>{});
#pragma unroll 1
        for (int r = 1; r + 1 < rounds; r += 2) {
            round(r, KwInt<1>{}, KwInt<1>{});
            round(r + 1, KwInt<0>{}, KwInt<1>{});
        }
        round(rounds - 1, KwInt<1>{}, KwInt<1>{});
#pragma unroll
        for (int y = 0; y < 8; ++y) column(prev, 0, y);
        output(prev, KwInt<1>{}, KwInt<0>{});
        kw_wait_copies<0>();                  // stages past the row's end are copied too, as zeros
        kw_barrier();

        // ---- the waves of a query tile become one: outputs side by side in LDS, 16-byte chunk c of query q at c XOR q ----
        l += __shfl_xor(l, 32);
        if (hi == 0) {
            red_m[wave][ql] = m;
            red_l[wave][ql] = l;
        }
        constexpr int QC = DV / 4;            // chunks of a query's output
        f32x4 *buf = reinterpret_cast<f32x4 *>(ring);
#pragma unroll
        for (int x = 0; x < DT; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                buf[(wave * 32 + ql) * QC + ((8 * x + 2 * i + hi) ^ (ql & (QC - 1)))] =
                    f32x4{o[x][4 * i], o[x][4 * i + 1], o[x][4 * i + 2], o[x][4 * i + 3]};
        kw_barrier();
        const bool whole = s0 == 0 && s1 == steps;
        const int slot = 2 * blockIdx.x + (u == u_begin ? 0 : 1);
        const int live = min(32 * WQ, grp.queries - tq0);
        for (int i = tid; i < live * QC; i += 64 * NW) {
            const int q = i / QC, c = i % QC, qi = q & 31;
            if (4 * c >= a.Dv) continue;
            float mq = red_m[q >> 5][qi], lq = 0.f;
#pragma unroll
            for (int x = 1; x < WK; ++x) mq = fmaxf(mq, red_m[x * WQ + (q >> 5)][qi]);
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < WK; ++x) {
                const int wv = x * WQ + (q >> 5);
                const float f = red_m[wv][qi] == -INFINITY ? 0.f : kp_weight(red_m[wv][qi], scale, mq);
                lq += red_l[wv][qi] * f;
                v += buf[(wv * 32 + qi) * QC + (c ^ (qi & (QC - 1)))] * f;
            }
            const size_t at = whole ? kv_query_row(a, first, h, tq0 + q) : (size_t)slot * a.tile_rows + q;
            float *ml = whole ? a.full_ml : a.part_ml;
            *reinterpret_cast<f32x4 *>((whole ? a.full_o : a.part_o) + at * a.Dv + 4 * c) = v;
            if (c == 0) {
                // the reference as a sequence's own part has it, to the bit
                ml[2 * at] = mq == -INFINITY ? mq : kv_scaled(a, flip ? -mq : mq);
                ml[2 * at + 1] = lq;
            }
        }
        __syncthreads();                      // the ring is free again
    }
}

// The group of sequence b among the groups (looked at by the whole wave): its
// first sequence, tiles, pages' steps and units, and the units before it and in
// all.
struct KpFound {
    int first, tiles, steps, units, before, total;
};
__device__ __forceinline__ KpFound kp_find(const AttnLaunch &pre, int b)
{
    const int lane = threadIdx.x & 63, G = pre.Hq / pre.Hkv;
    KpFound f{};
    for (int c = 0; c < pre.n_groups; c += 64) {
        const KpGroup g = kp_group(pre, min(c + lane, pre.n_groups - 1));
        const bool some = c + lane < pre.n_groups && g.queries > 0;
        const int n = some ? kv_shared(pre, min(g.first, pre.B - 1)) << pre.page_shift : 0;
        const int st = kv_units(n) * pre.Hkv * (some ? g.tiles : 0);
        const int incl = wave_scan_incl(st) + f.total;
        const uint64_t here = __ballot(some && g.first <= b && b < g.first + g.queries / G);
        if (here) {
            const int x = __ffsll((unsigned long long)here) - 1;
            f.before = __builtin_amdgcn_readlane(incl - st, x);
            f.first = __builtin_amdgcn_readlane(g.first, x);
            f.tiles = __builtin_amdgcn_readlane(g.tiles, x);
            const int pages = __builtin_amdgcn_readlane(n, x);
            f.steps = kv_steps(pages);
            f.units = kv_units(pages);
        }
        f.total = __builtin_amdgcn_readlane(incl, 63);
    }
    return f;
}

// Where the parts are that the shared pages left for query head qi of cache
// head h of sequence b (none where its own part holds all): row0 is the row of
// part_ml of the first, row1 + 2 w tile rows that of part w.
struct KpParts {
    int n, row0, row1;
};
__device__ __forceinline__ KpParts kp_parts(const AttnLaunch &pre, const KpFound &f, bool joined, int b, int h, int qi)
{
    KpParts p{};
    if (f.steps == 0 || !joined) return p;
    const int i = (b - f.first) * (pre.Hq / pre.Hkv) + qi, tile = i / pre.tile_rows, q = i - tile * pre.tile_rows;
    const int range = kv_range(pre, f.total), u0 = f.before + (h * f.tiles + tile) * f.units;
    // (groups that are no partition have sums past every range)
    const int w0 = min(max(u0 / range, 0), pre.n_wg - 1), w1 = min(max((u0 + f.steps - 1) / range, w0), pre.n_wg - 1);
    p.n = w1 - w0 + 1;
    p.row0 = (2 * w0 + (u0 == w0 * range ? 0 : 1)) * pre.tile_rows + q;
    p.row1 = 2 * w0 * pre.tile_rows + q;
    return p;
}
// Whether sequence b leaves its shared pages to its group.
__device__ __forceinline__ bool kp_joined(const AttnLaunch &own, int b)
{
    const int pages = kv_shared(own, b);
    return pages > 0 && kv_left(own, b) == pages;
}

// Joins the parts of `per` query heads of one sequence and cache head, the own
// parts first, then the shared pages'.  A wave looks up one head's parts and
// forms their factors; groups of threads then take every ng-th part, 4 columns
// a thread.
constexpr int SJ_HEADS = 4;                   // most heads of a workgroup

__global__ __launch_bounds__(KV_NT) void attn_shared_join_kernel(AttnLaunch own, AttnLaunch pre, int per)
{
    __shared__ __attribute__((aligned(16))) float red[KV_NT * 4];
    __shared__ float factor[SJ_HEADS][2 * KV_MAX_WG];
    __shared__ float inverse[SJ_HEADS];
    struct Parts {
        int n_own, n_pre;                     // 1: a row that is not cut, by its query
        int own0, own1, pre0, pre1;           // rows of part_ml: of the first part, and of the second less 2 tile rows a range
    };
    __shared__ Parts parts[SJ_HEADS];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int G = own.Hq / own.Hkv, chunks = (G + per - 1) / per;
    const int bh = blockIdx.x / chunks, b = bh / own.Hkv, h = bh - b * own.Hkv;
    const int i0 = (blockIdx.x - bh * chunks) * per, heads = min(per, G - i0);
    const size_t bq0 = (size_t)b * own.Hq + h * G + i0;
    const float *own_ml = own.part_ml, *own_full_ml = own.full_ml, *pre_ml = pre.part_ml, *pre_full_ml = pre.full_ml;

    if (wave < heads) {
        const int qi = i0 + wave;
        const size_t bq = bq0 + wave;
        Parts x{};
        int before, total;
        const KpFound grp = kp_find(pre, b);
        kv_prefix<KV_OWN>(own, b, &before, &total);
        const KvParts p = kv_parts<KV_OWN>(own, b, h * own.q_tiles + qi / own.tile_rows, before, total);
        x.n_own = p.steps == 0 ? 0 : p.w1 - p.w0 + 1;
        x.own0 = p.first * own.tile_rows + qi % own.tile_rows;
        x.own1 = 2 * p.w0 * own.tile_rows + qi % own.tile_rows;
        const KpParts pp = kp_parts(pre, grp, kp_joined(own, b), b, h, qi);
        x.n_pre = pp.n;
        x.pre0 = pp.row0;
        x.pre1 = pp.row1;
        const int n = x.n_own + x.n_pre, own_step = 2 * own.tile_rows, pre_step = 2 * pre.tile_rows;
        auto ml = [&](int w) -> const float * {
            if (w < x.n_own) return x.n_own == 1 ? own_full_ml + 2 * bq : own_ml + 2 * (size_t)(w == 0 ? x.own0 : x.own1 + w * own_step);
            w -= x.n_own;
            return x.n_pre == 1 ? pre_full_ml + 2 * bq : pre_ml + 2 * (size_t)(w == 0 ? x.pre0 : x.pre1 + w * pre_step);
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
            factor[wave][w] = f;
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) l += __shfl_xor(l, off);
        if (lane == 0) {
            parts[wave] = x;
            inverse[wave] = kv_inverse(l);
            kv_write_lse(own, bq, mx, l);
        }
    }
    __syncthreads();

    const int cols = own.Dv / 4, grp = tid / cols, col = tid - grp * cols;
    const int ng = KV_NT / cols / heads;      // groups a head (per is at most KV_NT / cols)
    const int v = grp / ng, sub = grp - v * ng;
    const bool mine = v < heads;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    if (mine) {
        const Parts x = parts[v];
        const size_t bq = bq0 + v;
        auto at = [&](size_t q) { return q * own.Dv + 4 * col; };
        auto add = [&](const float *part, const float *full, int n, int row0, int row1, int step, const float *f) {
            if (n == 1) {
                if (sub == 0) acc += *reinterpret_cast<const f32x4 *>(full + bq * own.Dv + 4 * col) * f[0];
                return;
            }
#pragma unroll 8
            for (int w = sub; w < n; w += ng)
                acc += *reinterpret_cast<const f32x4 *>(part + at((size_t)(w == 0 ? row0 : row1 + w * step))) * f[w];
        };
        add(own.part_o, own.full_o, x.n_own, x.own0, x.own1, 2 * own.tile_rows, factor[v]);
        add(pre.part_o, pre.full_o, x.n_pre, x.pre0, x.pre1, 2 * pre.tile_rows, factor[v] + x.n_own);
        *reinterpret_cast<f32x4 *>(red + 4 * tid) = acc;
    }
    __syncthreads();
    if (mine && sub == 0) {
        for (int x = 1; x < ng; ++x) acc += *reinterpret_cast<const f32x4 *>(red + 4 * (tid + x * cols));
        const float inv = inverse[v];
        const size_t to = (bq0 + v) * own.Dv + 4 * col;
        if (own.bf16)
            *reinterpret_cast<u32x2 *>((uint16_t *)own.out + to) =
                u32x2{pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv)};
        else *reinterpret_cast<f32x4 *>((float *)own.out + to) = acc * inv;
    }
}

// Joins the latent kernel's parts, whose lanes lie side by side: a workgroup
// takes 32 query heads of a sequence and COLS 32-column tiles, so that it reads
// whole lines of them.
template <int DV, int COLS>
__global__ __launch_bounds__(KV_NT) void attn_shared_wide_join_kernel(AttnLaunch own, AttnLaunch pre)
{
    constexpr int COL_SPLIT = DV / 32 / COLS, NF = KV_NT / 32;
    __shared__ float factor[2 * KW_MAX_WG + 2][32], red[NF][32];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, ql = lane & 31, hi = lane >> 5, grp = tid >> 5;
    const int G = own.Hq / own.Hkv, tiles = (G + 31) / 32;
    int at = blockIdx.x;
    const int cs = at % COL_SPLIT;
    at /= COL_SPLIT;
    const int q0 = at % tiles * 32;
    at /= tiles;
    const int h = at % own.Hkv, b = at / own.Hkv, nq = min(32, G - q0), qi = q0 + min(ql, nq - 1);
    const size_t bq = (size_t)b * own.Hq + h * G + qi;
    const KpFound f = kp_find(pre, b);
    int before, total;
    kv_prefix<KV_OWN>(own, b, &before, &total);
    const KvParts p = kv_parts<KV_OWN>(own, b, h * own.q_tiles + q0 / own.tile_rows, before, total);
    const KpParts pp = kp_parts(pre, f, kp_joined(own, b), b, h, qi);        // (a lane's own: tiles of a group may end among the heads)
    const int n_own = p.steps == 0 ? 0 : p.w1 - p.w0 + 1;
    int most = pp.n;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) most = max(most, __shfl_xor(most, off));
    const int n = n_own + most;
    // rows of the parts' references; of a row that is not cut its query's
    auto own_row = [&](int w) { return (size_t)p.slot(p.w0 + w) * own.tile_rows + qi % own.tile_rows; };
    auto pre_row = [&](int w) { return (size_t)(w == 0 ? pp.row0 : pp.row1 + 2 * w * pre.tile_rows); };
    auto ml = [&](int w, float &m, float &l) {
        m = -INFINITY;
        l = 0.f;
        if (w < n_own) {
            const float *x = n_own == 1 ? own.full_ml + 2 * bq : own.part_ml + 2 * own_row(w);
            m = x[0], l = x[1];
        } else if (w - n_own < pp.n) {
            const float *x = pp.n == 1 ? pre.full_ml + 2 * bq : pre.part_ml + 2 * pre_row(w - n_own);
            m = x[0], l = x[1];
        }
    };
    float mx = -INFINITY;
    for (int w = grp; w < n; w += NF) {
        float m, l;
        ml(w, m, l);
        mx = fmaxf(mx, m);
    }
    red[grp][ql] = mx;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < NF; ++x) mx = fmaxf(mx, red[x][ql]);
    __syncthreads();
    const float ref = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
    for (int w = grp; w < n; w += NF) {
        float m, l;
        ml(w, m, l);
        const float x = __builtin_amdgcn_exp2f(m - ref);
        sum += l * x;
        factor[w][ql] = x;
    }
    red[grp][ql] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int x = 0; x < NF; ++x) sum += red[x][ql];

    // wave i holds the i-th 8 columns of each tile: its lanes' are 8 i + 4 hi + 0..3
    f32x4 acc[COLS];
#pragma unroll
    for (int x = 0; x < COLS; ++x) acc[x] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto lanes = [&](size_t row) { return (row >> 5) * (32 * DV) + ((size_t)(cs * COLS * 4 + wave) * 64 + hi * 32 + (row & 31)) * 4; };
    auto add = [&](const float *part, const float *full, int n, int w, size_t row, float f) {
        if (n == 1) {
#pragma unroll
            for (int x = 0; x < COLS; ++x) {
                const int d = 32 * (cs * COLS + x) + 8 * wave + 4 * hi;
                if (d < own.Dv) acc[x] += *reinterpret_cast<const f32x4 *>(full + bq * own.Dv + d) * f;
            }
            return;
        }
        const float *src = part + lanes(row);
#pragma unroll
        for (int x = 0; x < COLS; ++x) acc[x] += *reinterpret_cast<const f32x4 *>(src + x * 1024) * f;
    };
#pragma unroll 4
    for (int w = 0; w < n_own; ++w) add(own.part_o, own.full_o, n_own, w, own_row(w), factor[w][ql]);
#pragma unroll 4
    for (int w = 0; w < most; ++w)
        if (w < pp.n) add(pre.part_o, pre.full_o, pp.n, w, pre_row(w), factor[n_own + w][ql]);
    if (ql >= nq) return;
    const float inv = kv_inverse(sum);
#pragma unroll
    for (int x = 0; x < COLS; ++x) {
        const int d = 32 * (cs * COLS + x) + 8 * wave + 4 * hi;
        if (d < own.Dv)
            *reinterpret_cast<u32x2 *>((uint16_t *)own.out + bq * own.Dv + d) =
                u32x2{pack_bf16(acc[x][0] * inv, acc[x][1] * inv), pack_bf16(acc[x][2] * inv, acc[x][3] * inv)};
    }
    if (cs == 0 && wave == 0 && hi == 0) kv_write_lse(own, bq, mx, sum);
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
        // More than two query tiles, and enough work that their reading the
        // pages once each counts for more than the LDS kernel's start and its
        // larger parts.  Whole calls, 8 cache heads, us with tiles / through
        // LDS: 48 queries a head, 128 wide, 512 positions 15 / 25, 4096 22 /
        // 27, 32768 74 / 47; 96 queries 4096 26 / 30; 160 queries 512 21 / 30,
        // 4096 36 / 36, 32768 113 / 69; 64 wide 160 queries 4096 26 / 28,
        // 32768 81 / 51; 256 wide 96 queries 4096 46 / 47, 32768 156 / 100.
        // Lengths and groups are on the device: the positions are the table's
        // room here and the queries the groups' mean, which is right for
        // tables as wide as their sequences and groups of like size.  48
        // queries behind 512 positions in a table of 16384 take 25 us, 160 take
        // 31 (tiles: 15 and 21); 160 behind 32768 beside 24 sequences that
        // share nothing keep the tiles (117; alone, through LDS, 68).
        const long work = (long)n_groups * Hkv * ((queries + KV_QT - 1) / KV_QT) * ((entries + KV_STEP - 1) / KV_STEP);
        if (bf16 && d <= 256 && queries > 32 && work >= 8192) {
            s.pre.wide = true;                // (tier: the widths, as above)
            const bool narrow = d <= 128 || (Dk <= 192 && Dv <= 128);        // (256-wide rows: four waves, all with queries of their own)
            s.pre.wq = !narrow ? 4 : queries <= 64 && d <= 128 ? 2 : queries <= 128 ? 4 : 8;
            s.pre.tile_rows = 32 * s.pre.wq;
            s.pre.n_wg = KW_MAX_WG;
            s.pre.min_units = KV_ROW_UNITS;
        }
    }
    s.own.q_tiles = (G + s.own.tile_rows - 1) / s.own.tile_rows;
    s.pre.q_tiles = 0;                        // each group's own
    return s;
}

// Own parts and shared pages of 16-head tiles in one launch: the shared pages'
// ranges first (four samples of one prompt: 8.4 and 7.9 us in two).  Two waves
// a SIMD up to 128-wide rows, whose ranges then run at once (fp32, 13 sequences
// of 12 heads of 80 in two groups behind 300 to 1999 positions: 21.9 us, with
// 300 registers and one wave 26.7).
template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(KV_NT, DK <= 128 ? 2 : 1) void attn_parts_kernel(AttnLaunch own, AttnLaunch pre)
{
    const int blk = (int)blockIdx.x - pre.n_wg;
    if (blk < 0) attn_rows<BF16, DK, DV, KV_WAVES, KV_PREFIX>(pre, blockIdx.x);
    else attn_rows<BF16, DK, DV, KV_WAVES, KV_OWN>(own, blk);
}
template <bool BF16, int DK, int DV, KvPart PART>
__global__ __launch_bounds__(KV_NT) void attn_part_kernel(AttnLaunch a)
{
    attn_rows<BF16, DK, DV, KV_WAVES, PART>(a, blockIdx.x);
}

// both: the shared pages too.
template <bool BF16, int DK, int DV>
static void launch_tile(const AttnLaunch &own, const AttnLaunch &pre, bool both, hipStream_t st)
{
    if constexpr (DK > 320) {                 // (two join buffers do not fit LDS)
        attn_part_kernel<BF16, DK, DV, KV_OWN><<<own.n_wg, KV_NT, 0, st>>>(own);
        attn_part_kernel<BF16, DK, DV, KV_PREFIX><<<pre.n_wg, KV_NT, 0, st>>>(pre);
    } else {
        if constexpr (BF16) {                 // (in fp32 always both)
            if (!both) return attn_part_kernel<BF16, DK, DV, KV_OWN><<<own.n_wg, KV_NT, 0, st>>>(own);
        }
        attn_parts_kernel<BF16, DK, DV><<<own.n_wg + pre.n_wg, KV_NT, 0, st>>>(own, pre);
    }
}

template <bool BF16>
static void launch_tiles(const AttnLaunch &own, const AttnLaunch &pre, const AttnPlan &p, bool both, hipStream_t st)
{
    if (p.tier == 64) launch_tile<BF16, 64, 64>(own, pre, both, st);
    else if (p.tier == 128) launch_tile<BF16, 128, 128>(own, pre, both, st);
    else if (p.tier == 256) launch_tile<BF16, 256, 256>(own, pre, both, st);
    else if constexpr (!BF16) {
        if (p.tier == 192) launch_tile<BF16, 192, 192>(own, pre, both, st);
        else if (p.tier == 320) launch_tile<BF16, 320, 256>(own, pre, both, st);
        else launch_tile<BF16, 576, 512>(own, pre, both, st);
    }
}

// Both parts of latent rows in one launch: the ring fills a CU's LDS, so the own
// parts' ranges follow where the shared pages leave CUs free (four sequences of
// 64 heads behind 2048 positions: 42 us, 57 in two; 32 behind 32768: 222, 226).
// Ranges of four units at least, not eight: 39 us there, but 16 sequences
// behind two prompts of 4096 70 for 53.
template <int DK, int DV, int WO, int WP, KwPast PAST>
__global__ __launch_bounds__(KV_NT) __attribute__((amdgpu_waves_per_eu(1, 1))) void attn_wide_parts_kernel(AttnLaunch own, AttnLaunch pre)
{
    const int blk = (int)blockIdx.x - pre.n_wg;
    if (blk < 0) attn_wide_rows<DK, DV, WP, PAST, KV_PREFIX>(pre, blockIdx.x);
    else attn_wide_rows<DK, DV, WO, PAST, KV_OWN>(own, blk);
}

template <int DK, int DV, int WO, int WP>
static void launch_wide(const AttnLaunch &own, const AttnLaunch &pre, hipStream_t st)
{
    const int n = own.n_wg + pre.n_wg;
    if (own.Dk == DK) attn_wide_parts_kernel<DK, DV, WO, WP, KW_NONE><<<n, KV_NT, 0, st>>>(own, pre);
    else if (own.Dk >= DV) attn_wide_parts_kernel<DK, DV, WO, WP, KW_TAIL><<<n, KV_NT, 0, st>>>(own, pre);
    else attn_wide_parts_kernel<DK, DV, WO, WP, KW_BOTH><<<n, KV_NT, 0, st>>>(own, pre);
}

// (a group has at least as many query heads as a sequence)
template <int DK, int DV>
static void launch_wide(const AttnLaunch &own, const AttnLaunch &pre, const SharedPlan &p, hipStream_t st)
{
    const int wo = p.own.wq, wp = p.pre.wq;
    if (wo == 4) launch_wide<DK, DV, 4, 4>(own, pre, st);
    else if (wo == 2 && wp == 4) launch_wide<DK, DV, 2, 4>(own, pre, st);
    else if (wo == 2) launch_wide<DK, DV, 2, 2>(own, pre, st);
    else if (wp == 4) launch_wide<DK, DV, 1, 4>(own, pre, st);
    else if (wp == 2) launch_wide<DK, DV, 1, 2>(own, pre, st);
    else launch_wide<DK, DV, 1, 1>(own, pre, st);
}

template <int DK, int DV, int NW>
static void launch_prefix(const AttnLaunch &a, int wq, hipStream_t st)
{
    if constexpr (NW == 8 && DK < 192) {      // (two stages a round: LDS does not hold three rounds of four)
        if (wq == 2) return attn_prefix_kernel<DK, DV, 2, 4><<<a.n_wg, 256, 0, st>>>(a);
    }
    if (wq == 4) attn_prefix_kernel<DK, DV, 4, NW><<<a.n_wg, 64 * NW, 0, st>>>(a);
    else if constexpr (NW == 8) attn_prefix_kernel<DK, DV, 8, NW><<<a.n_wg, 64 * NW, 0, st>>>(a);
}

hipError_t launch_attn_shared(const AttnLaunch &own, const AttnLaunch &pre, const SharedPlan &p, hipStream_t st)
{
    if (p.own.wide) {
        if (p.own.out_cols == 256) launch_wide<320, 256>(own, pre, p, st);
        else launch_wide<576, 512>(own, pre, p, st);
    } else {
        const bool both = !p.pre.wide;
        if (own.bf16) launch_tiles<true>(own, pre, p.own, both, st);
        else launch_tiles<false>(own, pre, p.own, both, st);
        if (both) {
        } else if (p.pre.tier == 64) launch_prefix<64, 64, 8>(pre, p.pre.wq, st);
        else if (p.pre.tier == 128) launch_prefix<128, 128, 8>(pre, p.pre.wq, st);
        else if (pre.Dk <= 192 && pre.Dv <= 128) launch_prefix<192, 128, 8>(pre, p.pre.wq, st);
        else launch_prefix<256, 256, 4>(pre, p.pre.wq, st);
    }
    const int G = own.Hq / own.Hkv;
    if (p.own.wide) {
        const int tiles = own.B * own.Hkv * ((G + 31) / 32);
        if (p.own.out_cols == 256) attn_shared_wide_join_kernel<256, 2><<<tiles * 4, KV_NT, 0, st>>>(own, pre);
        else attn_shared_wide_join_kernel<512, 2><<<tiles * 8, KV_NT, 0, st>>>(own, pre);
        return hipGetLastError();
    }
    // Heads of a workgroup: more share what is looked up, fewer are more workgroups.
    int per = SJ_HEADS;
    while (per > 1 && (per * (own.Dv / 4) > KV_NT || per > G || own.B * own.Hq / per < 512)) per /= 2;
    attn_shared_join_kernel<<<own.B * own.Hkv * ((G + per - 1) / per), KV_NT, 0, st>>>(own, pre, per);
    return hipGetLastError();
}

}  // namespace coli
