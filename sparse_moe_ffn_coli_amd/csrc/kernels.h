// kernels.h -- internal launch interface between the C ABI (api.hip) and the
// kernels (route.hip, ffn.hip, select.hip, attend.hip, shared.hip, kvcache.hip,
// plan.hip, rope.hip).  Not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace coli {

// Records caller-owned events between stages (instrumented entry points).
struct StageMarks {
    void *const *ev = nullptr;
    int n = 0;
    int next = 0;
    void mark(hipStream_t st)
    {
        if (ev && next < n && ev[next]) (void)hipEventRecord((hipEvent_t)ev[next], st);
        ++next;
    }
};

struct RouteLaunch {
    int T, D, E, K;
    bool bf16;
    const void *x;
    const void *wr;
    const float *bias;
    float *z;              // workspace [router_splits][T][E]: partial logits
    int32_t *tile_count;   // workspace [perm_tiles(T)][E]
    int32_t *done;         // workspace: counter of the fused top-K + permutation (zeroed by the router)
    int32_t *ids;
    float *w;
    int32_t *count, *offset, *perm, *inv;
    StageMarks *marks;     // nullable
};

struct FfnLaunch {
    int T, D, E, K, F;
    bool bf16;
    int bm;                // tile height of the grouped GEMMs (bf16)
    const void *x;
    const int32_t *ids;
    const float *w;
    const int32_t *count, *perm, *inv;
    const void *gate, *up, *down, *s_gate, *s_up, *s_down;
    bool use_int4;         // routed experts in int4 (then gate/up/down above are unused)
    const uint8_t *gate_q, *up_q, *down_q;
    const uint16_t *gate_s, *up_s, *down_s;
    int group;
    const float *residual;
    float *y;
    void *y_bf16;
    void *h;               // workspace [T*K + T][F] (bf16; fp16 in the int4 engine's chunk order for int4)
    uint16_t *x16;         // workspace [T][D] (int4 only): x in fp16, the int4 engine's chunk order
    void *o;               // workspace [T*K][D]
    float *sx;             // workspace [ksplit][T][D] (bf16 path): the shared expert's output (parts)
    int ksplit;            // parts of the down reduction (layers without routed rows; else 1)
    int4 *list_gu;         // workspace [ffn_max_tiles * ffn_col_tiles_gu] (256-row tiles)
    int4 *list_dn;         // workspace [ffn_max_tiles * ffn_col_tiles_dn] (256-row tiles)
    int32_t *n_items;      // workspace [20]: list lengths and per-XCD range starts
    StageMarks *marks;     // nullable
};

struct AttnLaunch {
    int B, Hq, Hkv, Dk, Dv;
    int page_shift, n_pages, max_pages;
    int cap;               // max_pages * page: the longest length
    bool bf16;
    const void *q, *k, *v; // v NULL: latent cache
    const int32_t *table, *lens, *idx;
    int idx_k;
    float scale_hi, scale_lo;   // scale * log2(e) in two floats
    float scale_cap;       // scores up to it times scale_lo are finite
    void *out;
    float *lse;            // nullable
    const float *acc_in;
    float *acc_out;        // nullable
    long ld;
    int q_tiles;           // query tiles per cache head (of groups: each has its own number)
    bool direct;           // a workgroup per row
    int n_wg, min_units;   // ranges of the main kernel (direct: rows); fewest steps in one
    float *part_o;         // workspace [2 n_wg][tile rows][Dv]: unnormalised parts
    float *part_ml;        // workspace [2 n_wg][tile rows][2]: their references and sums
    float *stats;          // workspace [B][Hq][2]: reference and 1 / sum (running weights only)
    float *scores;         // workspace [B][Hq][s_ld]: scores in units of log2 e (running weights only)
    long s_ld;
    // calls with shared pages only
    const int32_t *shared, *group_start;   // groups of sequences that share their first pages
    int n_groups;
    int tile_rows;         // query heads of a tile
    float *full_o;         // workspace [B][Hq][Dv]: unnormalised outputs of rows that are not cut
    float *full_ml;        // workspace [B][Hq][2]
    float scale_size;      // |scale_hi|
};

// Which kernel an attention call takes and how its workspace is laid out.
struct AttnPlan {
    bool wide;             // the LDS kernel
    int wq;                // its query tiles per workgroup
    int tile_rows, q_tiles;     // query heads a workgroup takes at a time, and how often per cache head
    int out_cols;          // columns of a part's rows
    int tier, waves;       // the other kernels' width and waves per workgroup
    bool direct;           // a workgroup per row, no parts
    int n_wg, min_units;
};

// The two parts of a call with shared pages.
struct SharedPlan {
    AttnPlan own, pre;
};

struct AppendLaunch {
    int B, Hkv, rows, page_shift, n_pages, max_pages, cap;
    int k_chunks, v_chunks;     // 16-byte chunks of a key and a value (0: latent)
    int tokens;                 // of a workgroup
    int first;                  // first row of the launch
    const void *k_new, *v_new;
    const int32_t *start, *table, *lens;
    void *k, *v;
};

struct EvictLaunch {
    int B, Hkv, page_shift, n_pages, max_pages, new_max_pages, cap;
    int k_chunks, v_chunks;
    void *k, *v;
    const int32_t *table, *lens;
    const float *acc;
    long ld;
    int keep, tail;
    const int32_t *new_table;
    int32_t *new_lens, *kept;
    float *new_acc;        // nullable
    long new_ld;
};

struct PlanLaunch {
    int B, page_shift, n_pages, max_pages, cap, rows;
    const int32_t *want, *shared;   // shared nullable
    int32_t *ring;
    const int32_t *state, *lens;
    int32_t *new_state, *new_lens;  // may be state and lens
    int32_t *table, *start, *slot, *pos;
};

struct RopeLaunch {
    int rows, nq, nk, nv;           // heads of each kind (0: absent)
    int Hkv, Dk, Dv;
    bool bf16;
    const void *q, *k, *v;
    long q_ld, k_ld, v_ld;          // elements from a token's row to the next
    const void *q_w, *k_w;          // nullable
    int width;                      // normed elements (0: none)
    float inv_width, eps;
    const double *freq;
    int rot, rot_at;                // rotated elements (0: none), first of them
    bool interleaved;
    float amp;
    const int32_t *pos, *slot;      // nullable
    void *q_out, *k_out, *pool_k, *pool_v;
    int page_shift, places;
    int heads, lane_shift;          // of a token, in all; log2 of the lanes of a head
    int first;                      // first token of the launch
    int tokens, parts, part_heads;  // tokens of a workgroup; workgroups that share them, and their heads
};

hipError_t launch_kv_plan(const PlanLaunch &a, hipStream_t st);
hipError_t launch_kv_rope(const RopeLaunch &a, hipStream_t st);
hipError_t launch_attn(const AttnLaunch &a, const AttnPlan &p, hipStream_t st);
hipError_t launch_attn_shared(const AttnLaunch &own, const AttnLaunch &pre, const SharedPlan &p, hipStream_t st);
SharedPlan attn_shared_plan(int B, int Hq, int Hkv, int Dk, int Dv, bool bf16, bool latent, int n_groups, int entries);
hipError_t launch_kv_append(const AppendLaunch &a, hipStream_t st);
hipError_t launch_kv_evict(const EvictLaunch &a, hipStream_t st);
AttnPlan attn_plan(int B, int Hq, int Hkv, int Dk, int Dv, bool bf16, bool latent, int entries);

hipError_t launch_route(const RouteLaunch &a, hipStream_t st);
// rows_per_len consecutive rows share an entry of lens; k may pass the 4096 of
// the public selection
hipError_t launch_index_topk(const float *scores, int rows, int L, long ld, const int32_t *lens, int rows_per_len,
                             int k, int tail, int32_t *idx, hipStream_t st);
hipError_t launch_ffn(const FfnLaunch &a, hipStream_t st);

int perm_tiles(int T);
int router_splits(int T, int D);
int ffn_tile_rows(int T, int E, int K, int int4);
long ffn_max_tiles(int T, int E, int K, int bm);
int ffn_col_tiles_gu(int F);
int ffn_col_tiles_dn(int D);
int ffn_down_splits(int T, int E, int D, int F, int bm);

}  // namespace coli
