// rope.hip -- queries and keys of new tokens on their way from the projection
// to the attention: each head's norm and the rotation by its position in one
// pass, the queries written side by side, keys and values straight to their
// places in the pages.
//   norm      x_i <- x_i w_i / sqrt(mean x^2 + eps)   over the head's first `width` elements
//   rotation  (x_i, x_j) <- (x_i c - x_j s, x_j c + x_i s),  c, s = amp (cos, sin)(pos freq)
// All in fp32, rounded once.  The angle is formed in 64 bits, as turns less
// whole turns: at position 2^24 an fp32 angle would be off by a radian.
//
// Bound by the bytes: every element is read and written once.  A head is held
// by a group of lanes, 16 bytes of it (bf16) each, so the norm's sum and the
// other half of a rotated pair are lane exchanges.  A workgroup takes one
// token, or several narrow ones, and works out their angles once for all
// heads, while the heads' first loads are on their way.
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

// E: elements of a lane.  NI: heads that a group of lanes has in flight.
template <bool BF16, int E, int NI>
__global__ __launch_bounds__(RP_NT) void kv_rope_kernel(RopeLaunch a)
{
    using Row = RopeRow<BF16, E>;
    constexpr int N = E / 4;                                 // groups of four elements, the half layout's unit
    constexpr size_t elt = BF16 ? 2 : 4;
    __shared__ __attribute__((aligned(16))) float angle[RP_PAIRS][2];
    const int tid = threadIdx.x, lanes = 1 << a.lane_shift;
    const int grp = tid >> a.lane_shift, lane = tid & (lanes - 1), groups = RP_NT >> a.lane_shift;
    const int e0 = lane * E;
    const int half = a.rot >> 1;
    const int parts = a.parts;                               // workgroups that share a block of tokens, by heads
    const int blk = blockIdx.x / parts, part = blockIdx.x - blk * parts;
    const int t0 = a.first + blk * a.tokens;
    const int nt = min(a.tokens, a.rows - t0);
    const int h_first = part * a.part_heads, h_n = min(a.part_heads, a.heads - h_first);
    const int items = nt * h_n;

    // A head of a token: where it comes from, whether the row counts.
    auto place = [&](int i, int &t, int &h) {
        const int x = a.tokens == 1 ? 0 : i / h_n;
        t = t0 + x;
        h = h_first + i - x * h_n;
    };
    auto source = [&](int t, int h) -> const char * {
        if (h < a.nq) return (const char *)a.q + ((size_t)t * a.q_ld + (size_t)h * a.Dk) * elt;
        h -= a.nq;
        if (h < a.nk) return (const char *)a.k + ((size_t)t * a.k_ld + (size_t)h * a.Dk) * elt;
        return (const char *)a.v + ((size_t)t * a.v_ld + (size_t)(h - a.nk) * a.Dv) * elt;
    };
    Row row[NI];
    auto load = [&](int i0) {
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int i = i0 + j * groups;
            int t, h;
            place(min(i, items - 1), t, h);
            if (i < items) row[j].load(source(t, h), e0, h < a.nq + a.nk ? a.Dk : a.Dv);
        }
    };
    load(grp);

    // the angles of the workgroup's tokens
    if (a.rot) {
        for (int i = tid; i < nt * half; i += RP_NT) {
            const int x = a.tokens == 1 ? 0 : i / half;
            const double turns = (double)a.pos[t0 + x] * (a.freq[i - x * half] * 0.15915494309189533577);
            float s, c;
            sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
            angle[i][0] = c * a.amp;
            angle[i][1] = s * a.amp;
        }
        __syncthreads();
    }

    const int h4 = half >> 2;
    for (int i0 = grp; i0 - grp < items; i0 += NI * groups) {     // (every lane takes part in the exchanges)
        if (i0 != grp) load(i0);
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int i = i0 + j * groups;
            if (i - grp >= items) break;
            int t, h;
            place(min(i, items - 1), t, h);
            const bool query = h < a.nq, key = !query && h < a.nq + a.nk;
            const int D = query || key ? a.Dk : a.Dv;
            const bool here = i < items && e0 < D && (!a.pos || a.pos[t] >= 0);
            float x[E];
            row[j].unpack(x);                                     // (what was not read meets nothing that is written)
            const void *w = query ? a.q_w : key ? a.k_w : nullptr;
            if (a.width) {
                float sum = 0.f;
                if (e0 < a.width) {
#pragma unroll
                    for (int e = 0; e < E; ++e) sum += E == 8 || e0 + (e & ~7) < a.width ? x[e] * x[e] : 0.f;
                }
                // (a value's head narrower than the norm: its sum is not used)
                for (int off = 1; off < lanes; off <<= 1) sum += __shfl_xor(sum, off);
                if (w && e0 < a.width) {
                    const float f = 1.f / sqrtf(sum * a.inv_width + a.eps);
#pragma unroll
                    for (int b = 0; b < E / 8; ++b) {             // (the width is whole eights)
                        if (e0 + 8 * b >= a.width) continue;
                        RopeRow<BF16, 8> part8;
                        part8.load(w, e0 + 8 * b, a.width);
                        float g8[8];
                        part8.unpack(g8);
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[8 * b + e] *= f * g8[e];
                    }
                }
            }
            if (a.rot) {
                const float *ang = &angle[(a.tokens == 1 ? 0 : t - t0) * half][0];
                if (a.interleaved) {
#pragma unroll
                    for (int b = 0; b < E / 8; ++b) {
                        const int at = e0 + 8 * b - a.rot_at;
                        if (at < 0 || at >= a.rot || !(query || key)) continue;
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const float c = ang[at + 2 * p], s = ang[at + 2 * p + 1];
                            const float u = x[8 * b + 2 * p], v = x[8 * b + 2 * p + 1];
                            x[8 * b + 2 * p] = u * c - v * s;
                            x[8 * b + 2 * p + 1] = v * c + u * s;
                        }
                    }
                } else {
                    // Group g of four elements meets group g +- h4, which another lane holds; which of its
                    // groups that is, is the same for all lanes that look the same way.
                    float up[E], down[E];
                    const int turn = h4 & (N - 1);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        up[e] = x[e];
                        down[e] = x[e];
                    }
                    if (turn & 1) {
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            up[e] = x[(e + 4) % E];
                            down[e] = x[(e + E - 4) % E];
                        }
                    }
                    if constexpr (N == 4) {
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
                        const int from_up = base + min(max(g + h4, 0) / N, lanes - 1);
                        const int from_down = base + max(g - h4, 0) / N;
                        float other[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float u = __shfl(up[4 * s + e], from_up), d = __shfl(down[4 * s + e], from_down);
                            other[e] = low ? u : d;
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
            if (w || (a.rot && (query || key))) row[j].pack(x);
            if (query) {
                row[j].store((char *)a.q_out + ((size_t)t * a.nq + h) * a.Dk * elt, e0, D);
                continue;
            }
            const int hk = h - a.nq - (key ? 0 : a.nk);
            if (key && a.k_out) row[j].store((char *)a.k_out + ((size_t)t * a.nk + hk) * a.Dk * elt, e0, D);
            const int at = a.slot ? a.slot[t] : -1;
            if (at < 0 || at >= a.places) continue;
            const size_t to = ((((size_t)(at >> a.page_shift) * a.Hkv + hk) << a.page_shift) + (at & ((1 << a.page_shift) - 1)));
            row[j].store((char *)(key ? a.pool_k : a.pool_v) + to * D * elt, e0, D);
        }
    }
}

template <bool BF16, int E>
static void launch_items(const RopeLaunch &a, int n_wg, int ni, hipStream_t st)
{
    if (ni == 1) kv_rope_kernel<BF16, E, 1><<<n_wg, RP_NT, 0, st>>>(a);
    else if (ni == 2) kv_rope_kernel<BF16, E, 2><<<n_wg, RP_NT, 0, st>>>(a);
    else kv_rope_kernel<BF16, E, 4><<<n_wg, RP_NT, 0, st>>>(a);
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
    const int per = (a.tokens * a.part_heads + groups - 1) / groups;
    const int ni = per <= 1 ? 1 : per <= 2 ? 2 : 4;
    const long all = (long)((a.rows + a.tokens - 1) / a.tokens);
    const long most = RP_MAX_WG / a.parts;
    for (long at = 0; at < all; at += most) {
        const long n = all - at < most ? all - at : most;
        a.first = (int)(at * a.tokens);
        const int n_wg = (int)(n * a.parts);
        if (a.bf16 && E == 8) launch_items<true, 8>(a, n_wg, ni, st);
        else if (a.bf16) launch_items<true, 16>(a, n_wg, ni, st);
        else if (E == 8) launch_items<false, 8>(a, n_wg, ni, st);
        else launch_items<false, 16>(a, n_wg, ni, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace coli
