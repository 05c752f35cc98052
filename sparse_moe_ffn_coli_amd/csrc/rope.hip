// rope.hip -- queries and keys of new tokens on their way from the projection
// to the attention: each head's norm and the rotation by its position in one
// pass, the queries written side by side, keys and values straight to their
// places in the pages.
//   norm      x_i <- x_i w_i / sqrt(mean x^2 + eps)   over the head's first `width` elements
//   rotation  (x_i, x_j) <- (x_i c - x_j s, x_j c + x_i s),  c, s = amp (cos, sin)(pos freq)
// All in fp32, rounded once.  The angle is formed in 64 bits, as turns less
// whole turns (at position 2^24 an fp32 angle would be off by a radian), and
// nothing of it is lost on the way to fp32 cosines and sines.
//
// Bound by the bytes: every element is read and written once.  A head is held
// by a group of lanes, 16 bytes of it (bf16) each, so the norm's sum and the
// other half of a rotated pair are lane exchanges.  A workgroup takes one
// token, or several narrow ones, and works out their angles once for all
// heads, while the heads' first loads are on their way.  A device copy moves
// 5.0 TB/s.
#include "device_common.h"
#include "kernels.h"

namespace coli {

constexpr int RP_NT = 256;
constexpr int RP_PAIRS = 2048;           // angles of a workgroup (16 KB of LDS)
constexpr int RP_MAX_WG = 1 << 22;       // workgroups of a launch: fewer than 2^32 threads

// E elements of a row from element e on, those past its width (whole eights)
// neither read nor written.
template <bool BF16, int E>
struct RopeRow {
    static constexpr int W = BF16 ? 1 : 2;                   // words of eight elements
    u32x4 w[W * E / 8];
    __device__ __forceinline__ void load(const void *row, int e, int width)
    {
#pragma unroll
        for (int i = 0; i < W * E / 8; ++i)
            if (e + i / W * 8 < width) w[i] = reinterpret_cast<const u32x4 *>((const char *)row + (size_t)e * 2 * W)[i];
    }
    __device__ __forceinline__ void store(void *row, int e, int width) const
    {
#pragma unroll
        for (int i = 0; i < W * E / 8; ++i)
            if (e + i / W * 8 < width) reinterpret_cast<u32x4 *>((char *)row + (size_t)e * 2 * W)[i] = w[i];
    }
    __device__ __forceinline__ void unpack(float (&x)[E]) const
    {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if constexpr (BF16) x[i] = __uint_as_float(i & 1 ? w[i / 8][i / 2 % 4] & 0xffff0000u : w[i / 8][i / 2 % 4] << 16);
            else x[i] = __uint_as_float(w[i / 4][i % 4]);
        }
    }
    __device__ __forceinline__ void pack(const float (&x)[E])
    {
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            if constexpr (BF16) {
                w[i / 8][i / 2 % 4] = (uint32_t)f32_to_bf16_bits(x[i]) | ((uint32_t)f32_to_bf16_bits(x[i + 1]) << 16);
            } else {
                w[i / 4][i % 4] = __float_as_uint(x[i]);
                w[i / 4][i % 4 + 1] = __float_as_uint(x[i + 1]);
            }
        }
    }
};

// The root's inverse: the hardware's, one ulp off, and the exact one where its
// argument could be no normal number.
__device__ __forceinline__ float rope_rsqrt(float x) { return x < 1e-30f ? 1.f / sqrtf(x) : __builtin_amdgcn_rsqf(x); }

// Value of the lane half a group further (the group's lanes are 2^LS).
template <int LS>
__device__ __forceinline__ float rope_across(float v)
{
    if constexpr (LS == 4) return __uint_as_float(__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0x128, 0xf, 0xf, false));   // a row of 16 turned by 8
    else return __shfl_xor(v, 1 << (LS - 1));
}

// E: elements of a lane.  LS: log2 of the lanes of a head (-1: any number of
// them, a.lane_shift), where LS >= 0 also means: one token a workgroup, whose
// angles a lane keeps in registers, and heads of E 2^LS elements that are normed
// and rotated whole or not at all, so that the other half of a pair is half a
// group of lanes away (16384 tokens of 32 + 8 + 8 heads of 128: 97 us, 403 MB at
// 4.2 TB/s; 164 by the general way).  A group of lanes has one head in flight
// (four: 103 us; workgroups of 512 threads: 131, of 128: 96).
template <bool BF16, int E, int LS>
__global__ __launch_bounds__(RP_NT) void kv_rope_kernel(RopeLaunch a)
{
    using Row = RopeRow<BF16, E>;
    constexpr int N = E / 4;                                 // groups of four elements, the half layout's unit
    constexpr bool WHOLE = LS >= 0;
    constexpr size_t elt = BF16 ? 2 : 4;
    __shared__ __attribute__((aligned(16))) float angle[WHOLE ? E << (WHOLE ? LS : 0) >> 1 : RP_PAIRS][2];
    const int lane_shift = WHOLE ? LS : a.lane_shift;
    const int tid = threadIdx.x, lanes = 1 << lane_shift;
    const int grp = tid >> lane_shift, lane = tid & (lanes - 1), groups = RP_NT >> lane_shift;
    const int e0 = lane * E;
    const int half = a.rot >> 1;
    const int parts = a.parts;                               // workgroups that share a block of tokens, by heads
    const int blk = parts == 1 ? blockIdx.x : blockIdx.x / parts, part = blockIdx.x - blk * parts;
    const bool one = WHOLE || a.tokens == 1;
    const int t0 = a.first + blk * a.tokens;
    const int nt = one ? 1 : min(a.tokens, a.rows - t0);
    const int h_first = part * a.part_heads, h_n = min(a.part_heads, a.heads - h_first);
    const int items = nt * h_n;

    // A head of a token: where it comes from, whether the row counts.
    auto place = [&](int i, int &t, int &h) {
        const int x = one ? 0 : i / h_n;
        t = t0 + x;
        h = h_first + i - x * h_n;
    };
    auto source = [&](int t, int h) -> const char * {
        if (h < a.nq) return (const char *)a.q + ((size_t)t * a.q_ld + (size_t)h * a.Dk) * elt;
        h -= a.nq;
        if (h < a.nk) return (const char *)a.k + ((size_t)t * a.k_ld + (size_t)h * a.Dk) * elt;
        return (const char *)a.v + ((size_t)t * a.v_ld + (size_t)(h - a.nk) * a.Dv) * elt;
    };
    // (of one token: where it goes, looked up before it is needed)
    const int pos_one = one && a.pos ? a.pos[t0] : 0, slot_one = one && a.slot ? a.slot[t0] : -1;
    Row row;
    auto load = [&](int i) {
        int t, h;
        place(min(i, items - 1), t, h);
        if (i < items) row.load(source(t, h), e0, h < a.nq + a.nk ? a.Dk : a.Dv);
    };
    load(grp);
    // the lane's weights, of queries and of keys
    Row w_q, w_k;
    if (a.q_w) w_q.load(a.q_w, e0, a.width);
    if (a.k_w) w_k.load(a.k_w, e0, a.width);

    // the angles of the workgroup's tokens
    if (a.rot) {
        for (int i = tid; i < nt * half; i += RP_NT) {
            const int x = one ? 0 : i / half;
            const double turns = (double)(one ? pos_one : a.pos[t0 + x]) * (a.freq[i - x * half] * 0.15915494309189533577);
            // half turns in fp32, and what that leaves as an angle: (c, s) turned by it
            const double halves = 2.0 * (turns - rint(turns));
            const float near = (float)halves, rest = (float)((halves - near) * 3.14159265358979323846);
            float s0, c0;
            sincospif(near, &s0, &c0);
            const float s = fmaf(c0, rest, s0), c = fmaf(-s0, rest, c0);
            angle[i][0] = c * a.amp;
            angle[i][1] = s * a.amp;
        }
        __syncthreads();
    }
    // the lane's angles (interleaved: the first half of them)
    float cs[WHOLE ? E : 1][2];
    if constexpr (WHOLE) {
        if (a.rot) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (a.interleaved && e >= E / 2) continue;
                const int at = a.interleaved ? e0 / 2 + e : (e0 & (E * lanes / 2 - 1)) + e;
                cs[e][0] = angle[at][0];
                cs[e][1] = angle[at][1];
            }
            if (!a.interleaved && lane < lanes / 2) {        // (x_i c - x_j s for the first half)
#pragma unroll
                for (int e = 0; e < E; ++e) cs[e][1] = -cs[e][1];
            }
        }
    }

    const int h4 = half >> 2;
    for (int i = grp; i - grp < items; i += groups) {        // (every lane takes part in the exchanges)
        if (i != grp) load(i);
        int t, h;
        place(min(i, items - 1), t, h);
        const bool query = h < a.nq, key = !query && h < a.nq + a.nk;
        const int D = query || key ? a.Dk : a.Dv;
        const bool here = i < items && e0 < D && (one ? pos_one : a.pos ? a.pos[t] : 0) >= 0;
        float x[E];
        row.unpack(x);                                     // (what was not read meets nothing that is written)
        const bool normed = query ? a.q_w != nullptr : key && a.k_w;
        if (a.width) {
            float sum = 0.f;
            if (WHOLE || e0 < a.width) {
#pragma unroll
                for (int e = 0; e < E; ++e) sum += E == 8 || e0 + (e & ~7) < a.width ? x[e] * x[e] : 0.f;
            }
            // (a value's head narrower than the norm: its sum is not used)
#pragma unroll
            for (int off = 1; off < (WHOLE ? 1 << (LS < 0 ? 0 : LS) : 64); off <<= 1)
                if (WHOLE || off < lanes) sum += __shfl_xor(sum, off);
            if (normed && (WHOLE || e0 < a.width)) {
                const float f = rope_rsqrt(sum * a.inv_width + a.eps);
                Row w;
#pragma unroll
                for (int e = 0; e < (int)(sizeof(w.w) / 16); ++e) w.w[e] = query ? w_q.w[e] : w_k.w[e];
                float g[E];
                w.unpack(g);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (E == 8 || e0 + (e & ~7) < a.width) x[e] *= f * g[e];   // (the width is whole eights)
            }
        }
        if (a.rot) {
            const float *ang = &angle[(one ? 0 : t - t0) * half][0];
            if (a.interleaved) {
#pragma unroll
                for (int b = 0; b < E / 8; ++b) {
                    const int at = e0 + 8 * b - a.rot_at;
                    if (!(query || key) || (!WHOLE && (at < 0 || at >= a.rot))) continue;
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const float c = WHOLE ? cs[WHOLE ? p : 0][0] : ang[at + 2 * p], s = WHOLE ? cs[WHOLE ? p : 0][1] : ang[at + 2 * p + 1];
                        const float u = x[8 * b + 2 * p], v = x[8 * b + 2 * p + 1];
                        x[8 * b + 2 * p] = u * c - v * s;
                        x[8 * b + 2 * p + 1] = v * c + u * s;
                    }
                }
            } else if constexpr (WHOLE) {
                float other[E];
#pragma unroll
                for (int e = 0; e < E; ++e) other[e] = rope_across<LS < 0 ? 4 : LS>(x[e]);
                if (query || key) {
#pragma unroll
                    for (int e = 0; e < E; ++e) x[e] = x[e] * cs[WHOLE ? e : 0][0] + other[e] * cs[WHOLE ? e : 0][1];
                }
            } else {
                // Group g of four elements meets group g +- h4, which another lane holds; which of its
                // groups that is, is the same for all lanes that look the same way (of two groups: for all).
                float up[E], down[E];
                const int turn = h4 & (N - 1);
#pragma unroll
                for (int e = 0; e < E; ++e) up[e] = turn & 1 ? x[(e + 4) % E] : x[e];
                if constexpr (N == 4) {
#pragma unroll
                    for (int e = 0; e < E; ++e) down[e] = turn & 1 ? x[(e + E - 4) % E] : x[e];
                    if (turn & 2) {
                        float u2[E], d2[E];
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            u2[e] = up[(e + 8) % E];
                            d2[e] = down[(e + E - 8) % E];
                        }
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            up[e] = u2[e];
                            down[e] = d2[e];
                        }
                    }
                }
                const int base = (tid & 63) & ~(lanes - 1);
#pragma unroll
                for (int s = 0; s < N; ++s) {
                    const int g = lane * N + s, at = 4 * g - a.rot_at;   // of the rotated part
                    const bool low = at < half;
                    const int from_up = base + min((g + h4) / N, lanes - 1), from_down = base + max(g - h4, 0) / N;
                    float other[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (N == 2) {
                            other[e] = __shfl(up[4 * s + e], low ? from_up : from_down);
                        } else {
                            const float u = __shfl(up[4 * s + e], from_up), d = __shfl(down[4 * s + e], from_down);
                            other[e] = low ? u : d;
                        }
                    }
                    if (at >= 0 && at < a.rot && (query || key)) {
                        const float *p = ang + 2 * (low ? at : at - half);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float c = p[2 * e], sn = p[2 * e + 1];
                            x[4 * s + e] = x[4 * s + e] * c + (low ? -other[e] : other[e]) * sn;
                        }
                    }
                }
            }
        }
        if (!here) continue;
        if (normed || (a.rot && (query || key))) row.pack(x);
        if (query) {
            row.store((char *)a.q_out + ((size_t)t * a.nq + h) * a.Dk * elt, e0, D);
            continue;
        }
        const int hk = h - a.nq - (key ? 0 : a.nk);
        if (key && a.k_out) row.store((char *)a.k_out + ((size_t)t * a.nk + hk) * a.Dk * elt, e0, D);
        const int at = one ? slot_one : a.slot ? a.slot[t] : -1;
        if (at < 0 || at >= a.places) continue;
        const size_t to = ((((size_t)(at >> a.page_shift) * a.Hkv + hk) << a.page_shift) + (at & ((1 << a.page_shift) - 1)));
        row.store((char *)(key ? a.pool_k : a.pool_v) + to * D * elt, e0, D);
    }
}

template <bool BF16>
static void launch_rope(const RopeLaunch &a, int E, bool whole, int n_wg, hipStream_t st)
{
    if (whole && a.lane_shift == 3) kv_rope_kernel<BF16, 8, 3><<<n_wg, RP_NT, 0, st>>>(a);
    else if (whole && a.lane_shift == 4) kv_rope_kernel<BF16, 8, 4><<<n_wg, RP_NT, 0, st>>>(a);
    else if (whole && a.lane_shift == 5) kv_rope_kernel<BF16, 8, 5><<<n_wg, RP_NT, 0, st>>>(a);
    else if (E == 8) kv_rope_kernel<BF16, 8, -1><<<n_wg, RP_NT, 0, st>>>(a);
    else kv_rope_kernel<BF16, 16, -1><<<n_wg, RP_NT, 0, st>>>(a);
}

hipError_t launch_kv_rope(const RopeLaunch &in, hipStream_t st)
{
    RopeLaunch a = in;
    a.heads = a.nq + a.nk + a.nv;
    if (a.rows == 0 || a.heads == 0) return hipSuccess;
    const int widest = a.Dv > a.Dk && a.nv ? a.Dv : a.Dk, E = widest > 512 ? 16 : 8;
    a.lane_shift = 0;
    while ((E << a.lane_shift) < widest) ++a.lane_shift;
    const int groups = RP_NT >> a.lane_shift;
    // Narrow tokens share a workgroup, the heads of few wide ones are spread
    // over several.
    a.tokens = 1;
    a.part_heads = a.heads;
    a.parts = 1;
    while (2 * a.tokens * a.heads <= 2 * groups && 2 * a.tokens * (a.rot / 2) <= RP_PAIRS && a.rows / (2 * a.tokens) >= 512)
        a.tokens *= 2;
    if (a.tokens == 1) {
        while (a.part_heads > groups && (long)a.rows * a.parts < 512) {
            a.part_heads = (a.part_heads + 1) / 2;
            a.parts = (a.heads + a.part_heads - 1) / a.part_heads;
        }
    }
    // Heads of 64, 128 or 256 elements, normed and rotated whole or not at all.
    const bool whole = a.tokens == 1 && a.Dk == E << a.lane_shift && (a.width == 0 || a.width == a.Dk) && (a.rot == 0 || a.rot == a.Dk);
    const long all = (long)((a.rows + a.tokens - 1) / a.tokens);
    const long most = RP_MAX_WG / a.parts;
    for (long at = 0; at < all; at += most) {
        const long n = all - at < most ? all - at : most;
        a.first = (int)(at * a.tokens);
        const int n_wg = (int)(n * a.parts);
        if (a.bf16) launch_rope<true>(a, E, whole, n_wg, st);
        else launch_rope<false>(a, E, whole, n_wg, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace coli
