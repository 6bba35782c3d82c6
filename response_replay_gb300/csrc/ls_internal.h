// ls_internal.h -- host-side interface between the C ABI (ls_api.cu) and the kernel
// translation units.  Not installed; the public interface is include/longstraw.h.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ls_sched.h"

// Bits of the per-device error word (see ls_last_device_error).
#define LS_DEVERR_CHECK 1u    // a device-side argument check failed
#define LS_DEVERR_TIMEOUT 2u  // a pipeline wait exceeded its time limit

// Counts every kernel launch the library makes (reported by ls_kernel_launches).
void ls_note_launch();

// Problem description shared by the replay-attention kernels (device pointers).
struct LsAttnArgs {
  const void* k_pool;        // bf16 [num_pages][hkv][ps][128]
  const void* v_pool;
  const int32_t* page_table; // [num_logical_pages]
  int32_t num_pages;
  int32_t ps_log2;           // page size = 1 << ps_log2
  int64_t P;                 // valid prompt tokens
  int32_t hkv, hq, g;        // g = hq / hkv
  int32_t pack;              // query rows per token in a tile: g (packed) or 1
  int32_t tiles;             // forward: query tiles per unit (2, or 1 when a packed unit's
                             // tokens all fit one tile)
  int32_t R;                 // response tokens (of each member)
  int32_t members;           // forward: responses of equal length R in one launch
  int32_t upm;               // units per member (INT32_MAX unless units are per member)
  int32_t rt;                // tokens the units cover: R, or members x R when the
                             // members' tokens are packed into shared tiles
  const void* q;             // bf16 [members][R][hq][128]
  const void* k_resp;        // bf16 [members][R][hkv][128]
  const void* v_resp;
  float scale_log2;          // softmax_scale * log2(e)
  float scale;               // softmax_scale
  uint32_t* err;             // device error word
};

struct LsFwdOut {
  void* o;                   // bf16 [members][R][hq][128]
  float* lse;                // [members][R][hq]
  float* part_o;             // workspace: [2*ctas][unit_rows][128]
  float* part_lse;           // workspace: [2*ctas][unit_rows]
};

struct LsBwdIn {
  const void* o;             // bf16 [R][hq][128]
  const float* lse;          // [R][hq]
  const void* d_o;           // bf16 [R][hq][128]
  float* delta;              // workspace [R][hq]: D = <dO, O>
  float* dt;                 // workspace [hq][rp]: D transposed, rp = R rounded up to 128
  float* lse2t;              // workspace [hq][rp]: lse log2(e) transposed
  float* dq;                 // [R][hq][128]
  float* dk;                 // [R][hkv][128]
  float* dv;
  float* part_dq;            // workspace: [pieces][unit_rows][128]
  float* part_dkdv;          // workspace: [2*ctas][2][128][128] (response-key kernel)
  int32_t accumulate;
  int32_t pair;              // dQ on CTA pairs (replay_bwd_dq_pair.cu) instead of one CTA
};

// Geometry of the replay kernels (fixed at build time).
int ls_fwd_unit_rows();
int ls_fwd_tile();
int ls_fwd_ctas_per_sm();
int ls_bwd_unit_rows();
int ls_bwd_tile();
int ls_bwd_ctas_per_sm();
int ls_num_units(int R, int hq, int hkv, int unit_rows);
// Forward: grouped-query packing factor (g for short responses, else 1) and units.
int ls_fwd_pack(int R, int hq, int hkv);
int ls_fwd_units(int R, int hq, int hkv);
int ls_fwd_tiles(int R, int hq, int hkv);
// Backward: the same packing for its one-tile units.
int ls_bwd_pack(int R, int hq, int hkv);
int ls_bwd_units(int R, int hq, int hkv);
// Backward dQ on CTA pairs: units of two tiles (one per CTA), their packing, and the
// number of pairs resident at once (the persistent grid).
int ls_bwd_pair_unit_rows();
int ls_bwd_pair_pack(int R, int hq, int hkv);
int ls_bwd_pair_units(int R, int hq, int hkv);
cudaError_t ls_bwd_pair_workers(int* pairs);

cudaError_t ls_launch_capture(const void* k, const void* v, void* k_pool, void* v_pool,
                              const int32_t* page_table, int32_t num_pages, int32_t ps_log2,
                              int32_t hkv, int64_t start_pos, int64_t n, int num_sms,
                              uint32_t* err, cudaStream_t st);

cudaError_t ls_launch_wait_timeout(uint32_t* err, cudaStream_t stream);
cudaError_t ls_launch_grpo_logp(const void* logits, bool is_bf16, int64_t T, int V,
                                const int32_t* targets, const float* ref_logp, float* logp_out,
                                float* lse_out, float* kl_out, uint32_t* err, int num_sms,
                                cudaStream_t stream);
cudaError_t ls_launch_validate_pages(const int32_t* page_table, int32_t num_logical,
                                     int32_t num_pages, uint32_t* seen, uint32_t* err,
                                     cudaStream_t st);

cudaError_t ls_launch_replay_fwd(const LsAttnArgs& a, const LsSched& sc, const LsFwdOut& out,
                                 cudaStream_t st);

cudaError_t ls_launch_bwd_dq(const LsAttnArgs& a, const LsSched& sc, const LsBwdIn& b,
                             cudaStream_t st);
// sc.ctas counts pairs here.
cudaError_t ls_launch_bwd_dq_pair(const LsAttnArgs& a, const LsSched& sc, const LsBwdIn& b,
                                  cudaStream_t st);

// Response-key dK / dV (tcgen05) and the bytes of its partial-sum workspace.
size_t ls_dkdv_part_bytes(int R, int hq, int hkv, int num_sms, const LsSegs* segs);
cudaError_t ls_launch_bwd_dkdv(const LsAttnArgs& a, const LsSegs& seg, const LsBwdIn& b,
                               int num_sms, cudaStream_t st);

cudaError_t ls_launch_replay_bwd(const LsAttnArgs& a, const LsSched& sc, const LsBwdIn& b,
                                 int num_sms, cudaStream_t st);

struct LsGrpoArgs {
  const void* logits;
  int32_t is_bf16;
  int64_t T;
  int32_t V;
  const int32_t* targets;
  const float* logp_old;
  const float* rewards;
  const int32_t* resp_lens;
  int32_t G, member_begin, member_end;
  float eps;
  double adv_eps;
  int32_t std_ddof;
  int32_t accumulate_loss;
  float* loss;
  void* dlogits;
  float* logp_out;
  float* stats;
  void* workspace;
  uint32_t* err;
};
size_t ls_grpo_ws_bytes(int64_t T, int G);
cudaError_t ls_launch_grpo(const LsGrpoArgs& a, int num_sms, cudaStream_t st);

// Gated-DeltaNet replay (gdn_replay.cu): head dims 128 (d_k = d_v), 64-token chunks.
struct LsGdnArgs {
  const float* state0;  // [H][128][128] (d_v x d_k): the captured state
  const void* q;        // bf16 [R][H][128]
  const void* k;
  const void* v;
  const float* g;       // [R][H] log decay
  const float* beta;    // [R][H]
  int32_t R, H;
  float scale;
  uint32_t* err;        // device error word (bounded pipeline waits report here)
};
size_t ls_gdn_ws_bytes(int R, int H, bool bwd);
cudaError_t ls_launch_gdn_fwd(const LsGdnArgs& a, void* o, float* state_out, void* ws,
                              cudaStream_t st);
cudaError_t ls_launch_gdn_bwd(const LsGdnArgs& a, const void* d_o, int accumulate, float* dq,
                              float* dk, float* dv, float* dg, float* dbeta, void* ws,
                              cudaStream_t st);

// Latent (MLA-style) replay forward (mla_replay.cu): rows of 576 bf16 values (512 latent
// + 64 rotary), outputs of 512; units = (128 token-major (t, h) rows) x (half of the
// output columns), unit u covering row tile u >> 1 and half u & 1.
struct LsMlaArgs {
  const void* pool;           // bf16 [num_pages][page_size][576]
  const int32_t* page_table;  // [ceil(P / page_size)]
  int32_t num_pages, ps_log2;
  int64_t P;
  const void* q;              // bf16 [R][H][576]
  const void* lat_resp;       // bf16 [R][576]
  int32_t R, H;
  float scale_log2;           // softmax scale x log2(e)
  void* o;                    // bf16 [R][H][512]
  float* lse;                 // [R][H]
  float* part_o;              // [pieces][128][256] partials of tail-unit pieces
  float* part_lse;            // [pieces][128]
  uint32_t* err;
};
int ls_mla_tile();
int ls_mla_unit_rows();
int ls_mla_half();
cudaError_t ls_launch_mla_fwd(const LsMlaArgs& a, const LsSched& sc, cudaStream_t st);
cudaError_t ls_launch_capture_latent(const void* src, void* pool, const int32_t* page_table,
                                     int32_t num_pages, int32_t ps_log2, int64_t start,
                                     int64_t n, int sms, uint32_t* err, cudaStream_t st);

// Latent replay backward (mla_replay_bwd.cu).
struct LsMlaBwdArgs {
  const void* pool;           // bf16 [num_pages][page_size][576]
  const int32_t* page_table;  // [ceil(P / page_size)]
  int32_t num_pages, ps_log2;
  int64_t P;
  const void* q;              // bf16 [R][H][576]
  const void* lat_resp;       // bf16 [R][576]
  const void* o;              // bf16 [R][H][512], the forward's output
  const float* lse;           // [R][H]
  const void* d_o;            // bf16 [R][H][512]
  int32_t R, H;
  float scale, scale_log2;
  float* delta;               // [R][H]: <dO, o>
  float* dq;                  // [R][H][576]
  float* dlat;                // [R][576]
  float* part_dq;             // [pieces][64][576] partials of tail-unit pieces
  float* part_dlat;           // [2 x d lat CTAs][128][320]
  uint32_t* err;
};
int ls_mla_bwd_tile();
int ls_mla_bwd_unit_rows();
int ls_mla_bwd_part_cols();
int ls_mla_bwd_dlat_ctas(int32_t R, int32_t H, int sms);
cudaError_t ls_launch_mla_bwd(const LsMlaBwdArgs& a, const LsSched& sc, int sms, cudaStream_t st);

// Query/key norm and rotary stage (qk_norm_rope.cu).  Rows are heads of 128 bf16 values;
// tensor i (0 queries, 1 keys, 2 values) has its rows at base + t * ts + h * hs elements.
struct LsRows {
  const void* p[3];   // values may be NULL
  int64_t ts[3], hs[3];
};
struct LsNormRopeArgs {
  int64_t T;
  int32_t hq, hkv;
  int32_t norm;              // 0: rotation only
  const void* w[2];          // norm weights of queries and keys, or NULL (ones)
  int32_t w_bf16;
  float w_offset, eps;
  const int32_t* pos;        // [axes][T]
  const double* inv_freq;    // [half], radians per position
  const int32_t* pair_axis;  // [half] or NULL (axis 0)
  int32_t axes, half, interleaved;
  uint32_t* err;
};
struct LsPoolDst {           // append: keys and values go to pages by slot
  void* k_pool;
  void* v_pool;
  const int32_t* slots;
  int32_t num_pages, ps_log2;
};
cudaError_t ls_launch_norm_rope_fwd(const LsNormRopeArgs& a, const LsRows& x, const LsRows& y,
                                    const LsPoolDst* dst, int sms, cudaStream_t st);
int ls_norm_rope_bwd_ctas(int64_t T, int sms);
// dy: gradients of the outputs (bf16 or fp32 rows); dw: fp32 [128] each or NULL; part:
// [ctas][2][128] fp32.
cudaError_t ls_launch_norm_rope_bwd(const LsNormRopeArgs& a, const LsRows& x, const LsRows& dy,
                                    int dy_bf16, const LsRows& dx, float* dwq, float* dwk,
                                    int accumulate, float* part, int sms, cudaStream_t st);

// Pages and slots of growing sequences (pages.cu).
struct LsExtendArgs {
  int32_t* table;            // [members][max_blocks]
  const int32_t* lens;
  const int32_t* add;        // NULL: all rows of every member in use
  const int32_t* free_list;
  const int32_t* used;
  int32_t* lens_out;
  int32_t* used_out;
  int32_t* added;            // [members] or NULL: what each got
  int32_t* slots;            // [capacity]
  int32_t* pos;              // [axes][capacity] or NULL
  int32_t members, max_blocks, num_free, num_pages, ps_log2, axes, pos0;
  int32_t rows;              // of every member (its tokens the last ones), 0: members packed
  int64_t capacity;
  uint32_t* err;
};
cudaError_t ls_launch_extend_pages(const LsExtendArgs& a, int sms, cudaStream_t st);

// Decode attention of a group over a shared prompt (decode_attn.cu).
struct LsDecodeArgs {
  const void* k_pool;        // prompt pages
  const void* v_pool;
  const int32_t* page_table;
  int32_t num_pages, ps_log2;
  int64_t P;
  const void* rk_pool;       // response pages
  const void* rv_pool;
  const int32_t* blocks;     // [members][max_blocks]
  const int32_t* lens;       // [members]
  int32_t r_num_pages, r_ps_log2, max_blocks;
  int32_t M, n, hq, hkv, g;
  const uint32_t* visible;   // trees: [M][n][words] rows that a row sees, NULL: the newest tokens in a line
  const int32_t* drafted;    // trees: [M] drafted tokens, or NULL (n)
  int32_t words;             // 32-bit words of a row of `visible`
  void* plan;                // trees of more than a tile of rows: how the work is cut (workspace)
  int32_t rts, cols;         // row tiles of 128 (token, head) rows; columns of rts CTAs each
  int32_t nt;                // prompt tiles of one KV head
  const void* q;             // bf16 [M][n][hq][128]
  float scale_log2;
  void* o;
  float* lse;
  float* part_o;             // [prompt slots][128][128], [response slots][n g, to 8][128], 8 rows together
  float* part_lse;           // same without the last dimension (log2 domain)
  uint32_t* err;
};
int ls_decode_row_tile();
int ls_decode_seg_tiles();  // tiles' worth of time that a segment of a response takes besides
// Rows of partial results: slots x rows.
int64_t ls_decode_prompt_rows(const LsDecodeArgs& a);
int64_t ls_decode_resp_rows(const LsDecodeArgs& a);
cudaError_t ls_launch_decode_attn(const LsDecodeArgs& a, cudaStream_t st);
// The same for trees of more rows than one tile a KV head (tree_attn.cu); cols: CTAs.
size_t ls_tree_plan_bytes(const LsDecodeArgs& a);
int64_t ls_tree_part_rows(const LsDecodeArgs& a);
cudaError_t ls_launch_tree_attn(const LsDecodeArgs& a, cudaStream_t st);

// Log probabilities of given tokens, entropies, top alternatives (token_logp.cu).
struct LsTokenLogpArgs {
  const void* logits;        // [T] rows of V values, ld apart
  int32_t is_bf16;
  int64_t T, ld;
  int32_t V;
  const int32_t* targets;    // [T] or NULL; -1: a padding row
  float temperature;
  int32_t top;               // alternatives, 0 to 32
  float* logp;               // [T] each, or NULL
  float* lse;
  float* entropy;
  float* top_logp;           // [T][top]
  int32_t* top_ids;
  void* workspace;           // parts' results, 16-byte aligned
  uint32_t* err;
};
struct LsTokenLogpBwdArgs {
  const void* logits;
  void* dlogits;
  int32_t is_bf16;
  int64_t T, ld, dld;
  int32_t V;
  const int32_t* targets;
  float temperature;
  int32_t top;
  const int32_t* top_ids;
  const float* lse;
  const float* entropy;
  const float* d_logp;
  const float* d_entropy;
  const float* d_top;
  uint32_t* err;
};
int ls_token_logp_parts(bool is_bf16, int64_t T, int V, int top, int sms);
size_t ls_token_logp_ws_bytes(int64_t T, int parts);
cudaError_t ls_launch_token_logp_fwd(const LsTokenLogpArgs& a, int parts, int sms, cudaStream_t st);
int64_t ls_token_logp_bwd_parts(const LsTokenLogpBwdArgs& a, int sms);
cudaError_t ls_launch_token_logp_bwd(const LsTokenLogpBwdArgs& a, int sms, cudaStream_t st);

// Drafted trees (drafts.cu).  Row r of member m is one of its n rows; its `drafted` nodes are
// the last of them, parents earlier rows of its own or -1.
struct LsDraftArgs {
  const int32_t* parents;    // [members][n]
  const int32_t* lens;       // [members], drafted tokens included
  const int32_t* drafted;    // [members] or NULL (n)
  int32_t members, n;
  uint32_t* err;
};
cudaError_t ls_launch_draft_tree(const LsDraftArgs& a, int32_t* visible, int32_t* positions,
                                 int32_t axes, int32_t pos0, cudaStream_t st);
cudaError_t ls_launch_accept_draft(const LsDraftArgs& a, const int32_t* tokens,
                                   const int32_t* chosen, int32_t* rows, int32_t* count,
                                   int32_t* follow, int32_t* ends, cudaStream_t st);
// Pages of one or several layers, layer l's pools l * stride values behind the first's.
struct LsLayerPools {
  void* k_pool;
  void* v_pool;
  int64_t stride;
  int32_t layers, num_pages, ps_log2, hkv;
};
cudaError_t ls_launch_compact_rows(const LsLayerPools& p, const int32_t* table, int32_t max_blocks,
                                   const LsDraftArgs& a, const int32_t* rows, const int32_t* count,
                                   cudaStream_t st);
cudaError_t ls_launch_copy_pages(const LsLayerPools& p, int32_t count, const int32_t* from,
                                 const int32_t* to, const int32_t* rows, uint32_t* err,
                                 cudaStream_t st);

// Pages given back and shared (pages.cu).
struct LsShareArgs {
  int32_t* table;            // [members][max_blocks]
  const int32_t* lens;
  int32_t* free_list;
  const int32_t* used;
  int32_t* shared;           // [num_pages] owners besides the first, or NULL
  int32_t* lens_out;
  int32_t* used_out;
  int32_t members, max_blocks, num_free, num_pages, ps_log2;
  uint32_t* err;
};
cudaError_t ls_launch_trim_pages(const LsShareArgs& a, const int32_t* new_lens, cudaStream_t st);
cudaError_t ls_launch_fork_pages(const LsShareArgs& a, const int32_t* src, const int32_t* keep,
                                 int32_t* copies, cudaStream_t st);
