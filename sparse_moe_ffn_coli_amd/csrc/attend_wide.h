// attend_wide.h -- the LDS kernel's statements (attend.h), of a function of
// <DK, DV, WQ, PAST, PART> with the launch `a`, the workgroup's number `blk` and
// in LDS `ring` (the stages), `rows_s` (their rows' addresses), `red_m` and
// `red_l` (the waves' references and sums).  Text and not a function: called
// from the kernel, with the launch by reference, the compiler reads all of it
// at the start and keeps it (32 sequences of 8000 to 32768 latent rows of 576,
// 128 heads: 286 us, 271 so).
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
    static_assert(sizeof(ring) == KW_RING * STAGE && KV_WAVES * OUT * 2 <= KW_RING * STAGE, "half of each wave's output fits the ring");

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);    // uniform: the copies' LDS addresses are
    const int qt = wave % WQ, kb = wave / WQ;
    const int G = a.Hq / a.Hkv;
    const int R = a.Hkv * a.q_tiles;
    KvRange rg;
    if (!kv_first<PART>(a, PART == KV_PREFIX ? 1 : R, rg, blk)) return;
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
        kv_next_row<PART>(a, R, b, n, steps, row);
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
        int h, q0, nq;                        // (nq: query heads of this wave's tile, may be none)
        if constexpr (PART == KV_PREFIX) {
            const KvTileOf t = kv_tile_of(a, b, row);
            h = t.h, q0 = t.q0 + 32 * qt, nq = t.queries - q0;
        } else {
            h = row / a.q_tiles, q0 = (row % a.q_tiles) * (32 * WQ) + 32 * qt;
            nq = G - q0;
        }
        const size_t qrow = (size_t)b * a.Hq + h * G + q0;
        const int len = PART == KV_ALL ? min(max(a.lens[b], 0), a.cap) : n;
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
                p[x] = PART == KV_ALL && a.idx ? a.idx[(size_t)b * a.idx_k + min(e, n - 1)] : e;
                p[x] = (e < end && p[x] >= 0 && p[x] < len) ? p[x] : -1;
            }
            int pg[PER];
#pragma unroll
            for (int x = 0; x < PER; ++x) {
                size_t entry = (size_t)(PART == KV_PREFIX ? kv_group_first(a, b) : b) * a.max_pages + (max(p[x], 0) >> a.page_shift);
                if constexpr (PART == KV_OWN) entry += kv_left(a, b);
                pg[x] = a.table[entry];
            }
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
            size_t query = qrow + ql;
            if constexpr (PART == KV_PREFIX) query = kv_query_row(a, kv_group_first(a, b), h, min(q0 + ql, q0 + max(nq, 1) - 1));
            const uint64_t rows = ql < nq ? (uint64_t)a.q + query * row_bytes : (uint64_t)kv_zeros;
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
                if (PART == KV_ALL && a.scores && ql < nq && t < seg) {
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
        const size_t slot = (size_t)(2 * blk + (u == u_begin ? 0 : 1)) * WQ + qt;
        f32x4 *part = reinterpret_cast<f32x4 *>(a.part_o + slot * OUT) + lane;
        uint16_t *out = (uint16_t *)a.out + (qrow + ql) * a.Dv;
        size_t query = qrow + ql;             // (groups: a row past the tile's queries is not written)
        if constexpr (PART == KV_PREFIX) query = kv_query_row(a, kv_group_first(a, b), h, q0 + ql);
        float *full = PART == KV_ALL ? nullptr : a.full_o + query * a.Dv;
        auto put = [&](int x, int i, f32x4 v) {
            if (!whole) {                     // a part: lanes side by side (attn_wide_join_kernel reads it the same way)
                part[(x * 4 + i) * 64] = v;
            } else if (PART != KV_ALL) {
                if (ql < nq && 32 * x + 8 * i + 4 * hi < a.Dv) *reinterpret_cast<f32x4 *>(full + 32 * x + 8 * i + 4 * hi) = v;
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
                if constexpr (PART == KV_ALL) kv_write_stats(a, qrow + ql, ma, la);
                else a.full_ml[2 * query] = ma, a.full_ml[2 * query + 1] = la;
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
                        } else if (PART != KV_ALL) {
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                bad |= 32 * x + 8 * i + 4 * hi < a.Dv && !(fabsf(full[32 * x + 8 * i + 4 * hi + c]) < INFINITY);
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
