/*
 * longstraw.h -- C ABI of the GB300 response-replay hot path.
 *
 * LongStraw trains GRPO at million-token contexts by evaluating the shared prompt once
 * without autograd, keeping only the state later tokens need (for full attention: K/V
 * pages), and replaying one response branch at a time under autograd (LongStraw paper
 * digest, "TL;DR" and "Method" steps 1-4; explainer "LongStraw: fitting million-token
 * RL onto a fixed GPU budget", "The move: change the graph boundary" and "Serial replay
 * makes G a schedule").  This library is that replay for one full-attention layer plus
 * the GRPO loss, on one GPU:
 *
 *   ls_capture_kv          write the prompt's K/V into pages behind a page table
 *   ls_replay_attn_fwd     exact attention of one response branch over the captured
 *                          pages plus causal self-attention, split-KV partials merged
 *                          by log-sum-exp
 *   ls_replay_attn_bwd     dQ through prompt and response keys; dK/dV for the
 *                          response's own keys only (the prompt state is stopgrad)
 *   ls_grpo_loss_fwd_bwd   token-level clipped surrogate with group-relative
 *                          advantages and its logits gradient
 *   ls_mla_replay_fwd      the forward over latent (MLA-style) pages, which may be
 *                          held in host memory
 *   ls_mla_replay_bwd      its backward: dq, and the gradient of the response's own
 *                          latent rows (the prompt rows are stopgrad)
 *   ls_qk_norm_rope_*      the stage between a layer's projections and its attention:
 *                          query / key norms with rotary positions, forward, backward,
 *                          and fused with the write into pages
 *   ls_extend_pages        pages and slots of a group's growing responses, packed or
 *                          (_by_member) in every member's own rows
 *   ls_extend_drafts       the same for drafted tokens: also how many each member got
 *   ls_decode_attn         the rollout's decode step: every member's newest tokens over
 *                          the shared captured prompt and its own paged response
 *   ls_draft_tree, ls_decode_attn_tree, ls_accept_draft, ls_compact_rows
 *                          the decode step over a tree of drafted tokens a member: its plan,
 *                          its attention, the accepted path, and that path's keys and values
 *                          moved together
 *   ls_trim_pages, ls_fork_pages, ls_copy_pages
 *                          pages given back, and shared by branches of a response
 *   ls_token_logp_*        log probabilities of given tokens, entropies and top alternatives
 *                          of vocabulary rows, and their backward
 *
 * Conventions shared by every call
 *   - Memory: every pointer argument is DEVICE memory on the current CUDA device unless
 *     stated otherwise, allocated and owned by the caller.  The library allocates no
 *     device memory; temporary space is the caller's `workspace` (size from the
 *     matching *_workspace query, which depends on the current device's SM count).
 *   - Streams: work is enqueued on `stream` (NULL = legacy default stream) and the
 *     calls return without synchronising, except ls_last_device_error.
 *   - Layouts: dense row-major, innermost dimension last, no padding.  bf16 is the
 *     upper half of an IEEE-754 binary32 (1 sign, 8 exponent, 7 fraction bits);
 *     fp32 is binary32.
 *   - Alignment: every device pointer must be 16-byte aligned, except the per-token
 *     arrays of the loss and scoring calls (targets, logp_old, ref_logp, logp_out,
 *     lse_out, kl_out), which need 4 bytes, so that a member's slice of a token-major
 *     buffer can be passed whatever its token offset, and the index arrays of the
 *     query / key stage and of the decode step (4 bytes, inv_freq 8, unless said
 *     otherwise there).
 *   - Errors: arguments are checked on the host first; on failure the call returns
 *     LS_ERR_INVALID_ARG / LS_ERR_UNSUPPORTED / LS_ERR_WORKSPACE and launches
 *     nothing.  A failed launch returns LS_ERR_CUDA.  Conditions only the device can
 *     see (a page id outside the pool, response lengths that do not add up, a
 *     pipeline wait that exceeded its time limit) never trap: the kernel skips the
 *     offending access, records a code in a per-device error word and carries on;
 *     ls_last_device_error() reports and clears it.
 *   - Determinism: no floating-point atomics; the same inputs and launch
 *     configuration give bit-identical outputs.
 *   - Device reset: the library looks up the device addresses of its own device
 *     variables (the error word, the no-alloc scratch) once per device and keeps them
 *     for the life of the process.  cudaDeviceReset() unloads the library's device
 *     image, so these addresses go stale: do not call the library on a device after
 *     resetting it in the same process.
 */
#ifndef LONGSTRAW_H
#define LONGSTRAW_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* ls_stream_t;

typedef enum {
  LS_OK = 0,
  LS_ERR_INVALID_ARG = 1,   /* a size, pointer, alignment or dtype is not accepted   */
  LS_ERR_UNSUPPORTED = 2,   /* valid in principle, not built (e.g. head_dim != 128)  */
  LS_ERR_WORKSPACE = 3,     /* workspace NULL or smaller than the query says          */
  LS_ERR_CUDA = 4,          /* a CUDA runtime/driver call failed                      */
  LS_ERR_TIMEOUT = 5,       /* a device pipeline wait hit its time limit              */
  LS_ERR_DEVICE_CHECK = 6   /* a device-side argument check failed (bad page id ...)  */
} ls_status;

typedef enum { LS_BF16 = 0, LS_FP32 = 1 } ls_dtype;

/* The captured prompt state of one attention layer: K and V pages plus the page table
 * (the digest's "CP-sharded KV pages" of the Qwen implementation, held whole on one
 * GPU).  Caller-owned; read-only after capture.
 *   k_pool, v_pool  bf16 [num_pages][num_kv_heads][page_size][head_dim]
 *   page_table      int32 [num_logical_pages]: logical page -> physical page in
 *                   [0, num_pages).  Logical page p holds prompt positions
 *                   [p * page_size, (p + 1) * page_size).
 *   num_tokens      P, the valid prompt positions; P <= num_logical_pages * page_size.
 *                   Positions >= P on the last page are never read by attention.
 * Supported: head_dim == 128; page_size a power of two in [16, 4096]; num_pages *
 * num_kv_heads * page_size < 2^31.
 * The pools may live in host memory that the GPU reads directly (pinned, mapped
 * allocations; on a Grace-Blackwell node the Grace memory behind NVLink-C2C): the
 * capture writes and every replay reads them there, with no staging copy.  This is the
 * GB300 counterpart of holding the prompt's pages in CPU memory (explainer, "Two
 * incompatible architectures", GLM bullet).  page_table stays in GPU memory. */
typedef struct {
  void* k_pool;
  void* v_pool;
  const int32_t* page_table;
  int32_t num_pages;
  int32_t num_logical_pages;
  int32_t page_size;
  int32_t num_kv_heads;
  int32_t head_dim;
  int64_t num_tokens;
} ls_kv_cache;

/* ---------------------------------------------------------------- capture
 * Prompt capture keeps the prompt's K/V as resident pages (digest, Method step 1;
 * explainer, "The move: change the graph boundary").  Copies positions
 * [start_pos, start_pos + n) of the prompt:
 *   k_pool[pt[p / ps]][h][p % ps][:] = k[p - start_pos][h][:]   (same for v)
 * k, v: bf16 [n][num_kv_heads][head_dim].  Bit copy.  Can be called in chunks.  A page
 * id outside [0, num_pages) skips that position and sets LS_ERR_DEVICE_CHECK.
 * start_pos + n must not exceed num_logical_pages * page_size. */
ls_status ls_capture_kv(const ls_kv_cache* cache, const void* k, const void* v,
                        int64_t start_pos, int64_t n, ls_stream_t stream);

/* ---------------------------------------------------------------- replay forward
 * Exact attention of one response branch (explainer, "Serial replay makes G a
 * schedule"; digest, Method step 3) over the captured prompt and causally over its own
 * keys; the prompt's split-KV partials are composed by log-sum-exp into the exact
 * output, which the pages do across eight GPUs (explainer, "Two incompatible
 * architectures", Qwen bullet) and this call does on one:
 *   s_{t,j} = softmax_scale * <q_{t,h}, k_{j,h/g}>,  j over all P prompt positions and
 *             response positions j <= t (g = Hq / num_kv_heads)
 *   lse_{t,h} = log sum_j exp(s_{t,j})           (natural log)
 *   o_{t,h}   = sum_j exp(s_{t,j} - lse_{t,h}) v_j
 * q: bf16 [R][Hq][128]; k_resp, v_resp: bf16 [R][num_kv_heads][128] (the response's
 * own keys/values); o: bf16 [R][Hq][128] (round-to-nearest-even); lse: fp32 [R][Hq].
 * num_splits (>= 1) cuts the prompt into that many contiguous ranges of 128-token
 * tiles; the result does not depend on it beyond rounding.  Hq % num_kv_heads == 0.
 * softmax_scale must be finite and > 0 (typically 1/sqrt(128)).
 * R == 0 is a no-op.  P == 0 is plain causal attention of the response. */
ls_status ls_replay_attn_fwd_workspace(const ls_kv_cache* cache, int R, int Hq,
                                       int num_splits, size_t* bytes);
ls_status ls_replay_attn_fwd(const ls_kv_cache* cache, const void* q, const void* k_resp,
                             const void* v_resp, int R, int Hq, float softmax_scale,
                             int num_splits, void* o, float* lse, void* workspace,
                             size_t workspace_bytes, ls_stream_t stream);

/* ls_replay_attn_fwd_members: the same forward for `members` responses of equal length
 * R over the same captured prompt, in one launch.  Pre-step scoring runs every member
 * of a group forward-only before the step (explainer, "Serial replay makes G a
 * schedule": the response branches share the read-only prompt state); batching them
 * lets the members' rows that share a KV head walk each prompt K/V tile together, so
 * the prompt streams from HBM about once for all of them instead of once per member.
 * Member m's rows see the whole prompt and member m's own response keys (j <= t)
 * only; its result equals ls_replay_attn_fwd on member m's slices (up to rounding).
 * q: bf16 [members][R][Hq][128]; k_resp, v_resp: bf16 [members][R][num_kv_heads][128];
 * o: bf16 [members][R][Hq][128]; lse: fp32 [members][R][Hq].  Short responses (the
 * grouped-query-packed regime) pack the members' tokens into shared 128-row tiles, so
 * one K/V tile serves members x g x R rows; there a member's rows also meet the other
 * members' response keys, masked to zero weight, so inputs must be finite (a non-finite
 * value times a zero weight is not zero; the one-response call has the same property
 * for the causally masked keys of its own response).  members >= 0 (0 or R == 0 is a
 * no-op); LS_ERR_UNSUPPORTED when members x R or the work-unit count exceeds 2^30.
 * Other arguments and errors as ls_replay_attn_fwd; ls_replay_attn_fwd is this call
 * with members = 1. */
ls_status ls_replay_attn_fwd_members_workspace(const ls_kv_cache* cache, int R, int members,
                                               int Hq, int num_splits, size_t* bytes);
ls_status ls_replay_attn_fwd_members(const ls_kv_cache* cache, const void* q, const void* k_resp,
                                     const void* v_resp, int R, int members, int Hq,
                                     float softmax_scale, int num_splits, void* o, float* lse,
                                     void* workspace, size_t workspace_bytes,
                                     ls_stream_t stream);

/* ---------------------------------------------------------------- replay backward
 * Gradient of the replayed branch with the prompt state stopgrad: only
 * d(loss)/d(theta) at the captured state is formed and the path through the prompt
 * state is dropped (digest, Method, last paragraph; explainer, Figure 2 caption), so
 * prompt keys and values receive no gradient and only the response's own keys do
 * (explainer, "Two incompatible architectures": K/V gradient pages exist only where a
 * response backward touches them).  With P_{t,j} = exp(s_{t,j} - lse_t),
 * D_t = <dO_t, O_t>, dS_{t,j} = P_{t,j} (<dO_t, v_j> - D_t):
 *   dq_t   = softmax_scale * sum_j dS_{t,j} k_j          (prompt and response keys)
 *   dk_j   = softmax_scale * sum_{h in group, t >= j} dS_{t,j} q_t    (response j)
 *   dv_j   = sum_{h in group, t >= j} P_{t,j} dO_t                    (response j)
 * o, lse: the forward's outputs for the same inputs; d_o: bf16 [R][Hq][128].
 * dq: fp32 [R][Hq][128]; dk_resp, dv_resp: fp32 [R][num_kv_heads][128].
 * accumulate != 0 adds into dq/dk_resp/dv_resp instead of overwriting them (serial
 * replay accumulates gradients member by member: digest, Method step 3).
 * The environment variable LS_BWD_PAIR=1, read once per process, runs dQ on pairs of
 * SMs (cluster CTA pairs); the default one-CTA kernel measured faster on every shape
 * tried.  Both give the same results up to summation order; the workspace query and
 * the call must see the same setting. */
ls_status ls_replay_attn_bwd_workspace(const ls_kv_cache* cache, int R, int Hq,
                                       int num_splits, size_t* bytes);
ls_status ls_replay_attn_bwd(const ls_kv_cache* cache, const void* q, const void* k_resp,
                             const void* v_resp, const void* o, const float* lse,
                             const void* d_o, int R, int Hq, float softmax_scale,
                             int num_splits, int accumulate, float* dq, float* dk_resp,
                             float* dv_resp, void* workspace, size_t workspace_bytes,
                             ls_stream_t stream);

/* ---------------------------------------------------------------- ragged members
 * ls_replay_attn_fwd_ragged / ls_replay_attn_bwd_ragged: the replay of `members`
 * responses of different lengths lens[0 .. members) (a HOST array) over the same captured
 * prompt, in one forward and one backward launch.  The members' tokens lie back to back
 * (member m's token t is row off_m + t, off_m = lens[0] + ... + lens[m-1], T = the sum):
 *   q, o, d_o: bf16 [T][Hq][128]; k_resp, v_resp: bf16 [T][num_kv_heads][128];
 *   lse: fp32 [T][Hq]; dq: fp32 [T][Hq][128]; dk_resp, dv_resp: fp32 [T][num_kv_heads][128].
 * Each member sees the whole prompt and its own response keys j <= t only (a
 * block-diagonal causal mask over the concatenation), so member m's results equal the
 * one-response calls on its slices, up to rounding; the work of all members shares one
 * schedule over the GPU (the pages replay members one by one; on one GPU with room for
 * a whole group this fills the SMs better for short and mixed lengths).  As for the
 * batched forward, inputs must be finite: a member's rows meet other members' keys with
 * zero weight, and a non-finite value times zero is not zero.
 * 1 <= members <= 64, lens[m] >= 0 (empty members allowed); T <= 2^30, and for the
 * backward of more than one member T <= 131,072 (LS_ERR_UNSUPPORTED otherwise).  Other
 * arguments, workspace and errors as ls_replay_attn_fwd / ls_replay_attn_bwd, which are
 * these calls with one member. */
ls_status ls_replay_attn_fwd_ragged_workspace(const ls_kv_cache* cache, const int32_t* lens,
                                              int members, int Hq, int num_splits, size_t* bytes);
ls_status ls_replay_attn_fwd_ragged(const ls_kv_cache* cache, const void* q, const void* k_resp,
                                    const void* v_resp, const int32_t* lens, int members, int Hq,
                                    float softmax_scale, int num_splits, void* o, float* lse,
                                    void* workspace, size_t workspace_bytes, ls_stream_t stream);
ls_status ls_replay_attn_bwd_ragged_workspace(const ls_kv_cache* cache, const int32_t* lens,
                                              int members, int Hq, int num_splits, size_t* bytes);
ls_status ls_replay_attn_bwd_ragged(const ls_kv_cache* cache, const void* q, const void* k_resp,
                                    const void* v_resp, const void* o, const float* lse,
                                    const void* d_o, const int32_t* lens, int members, int Hq,
                                    float softmax_scale, int num_splits, int accumulate, float* dq,
                                    float* dk_resp, float* dv_resp, void* workspace,
                                    size_t workspace_bytes, ls_stream_t stream);

/* ---------------------------------------------------------------- GRPO loss
 * The clipped surrogate of the digest's Method section,
 *   L = -(1/G) sum_i (1/R_i) sum_t min(rho_{i,t} A_i, clip(rho_{i,t}, 1-eps, 1+eps) A_i),
 *   rho = exp(logp - logp_old),  logp = logits[target] - logsumexp(logits),
 *   A_i = (r_i - mean r) / (std r + adv_eps)   (group-relative; std with std_ddof;
 *                                             mean/std in fp64),
 * and its gradient dL/dlogits_v = c_t (1[v == target] - softmax_v), where
 * c_t = -A_i rho_t / (G R_i) when the unclipped term is the active minimum (ties
 * included) and 0 when the clip holds the term constant.
 * Serial replay calls this once per member (digest, Method step 3): logits hold the
 * tokens of members [member_begin, member_end) back to back (member-major), while
 * rewards and resp_lens describe all G members so every call sees the whole group.
 *   logits   [T][V] of type dtype; T = sum of resp_lens over the range (checked on the
 *            device: a mismatch sets LS_ERR_DEVICE_CHECK and writes nothing)
 *   targets  int32 [T] in [0, V);  logp_old fp32 [T]
 *   rewards  fp32 [G];  resp_lens int32 [G]
 *   loss     fp32 device scalar: this call's contribution (accumulate_loss != 0 adds
 *            it to the current value)
 *   dlogits  [T][V] of type dtype (may alias nothing else)
 *   logp_out fp32 [T] or NULL
 *   stats    fp32 [4] or NULL: {tokens whose gradient the clip zeroed, sum of rho,
 *            min rho, max rho} over this call's tokens
 * G - std_ddof must be >= 1; 0 <= member_begin <= member_end <= G; V <= 2^30. */
ls_status ls_grpo_workspace(int64_t T, int G, size_t* bytes);
ls_status ls_grpo_loss_fwd_bwd(const void* logits, ls_dtype dtype, int64_t T, int V,
                               const int32_t* targets, const float* logp_old,
                               const float* rewards, const int32_t* resp_lens, int G,
                               int member_begin, int member_end, float eps, float adv_eps,
                               int std_ddof, int accumulate_loss, float* loss, void* dlogits,
                               float* logp_out, float* stats, void* workspace,
                               size_t workspace_bytes, ls_stream_t stream);

/* ls_grpo_loss_fwd_bwd_noalloc: the same computation as ls_grpo_loss_fwd_bwd, for
 * callers that cannot provide or allocate device memory at the point of the call (for
 * example a training loop whose host framework plans all device memory up front and
 * forbids new allocations mid-step).  The paper has no counterpart: this is an
 * interface convenience of this library.  Instead of a caller workspace it uses one
 * fixed scratch array inside the library's device image (4.125 MiB per device, held
 * until process exit); it calls no allocator.  Limits: T <= 262,144 tokens and
 * G <= 1,024 members, otherwise LS_ERR_WORKSPACE is returned and nothing is launched.
 * The first call on a device looks up the array's device address (a runtime query,
 * no allocation); make that first call before any stream capture.  All calls share
 * the array: calls whose kernels could overlap on the GPU race, so order them (one
 * stream, or events).  Nothing in the array needs to start at zero.  Arguments and
 * outputs otherwise as ls_grpo_loss_fwd_bwd. */
ls_status ls_grpo_loss_fwd_bwd_noalloc(const void* logits, ls_dtype dtype, int64_t T, int V,
                                       const int32_t* targets, const float* logp_old,
                                       const float* rewards, const int32_t* resp_lens, int G,
                                       int member_begin, int member_end, float eps,
                                       float adv_eps, int std_ddof, int accumulate_loss,
                                       float* loss, void* dlogits, float* logp_out,
                                       float* stats, ls_stream_t stream);

/* ls_grpo_logp: pre-step scoring without a gradient (LongStraw explainer: the replay
 * is the gradient pass of one member; the log-probabilities a step needs before it,
 * logp_old and a reference policy's, come from forward-only passes like this one).
 *   logp_t = logits[t][targets[t]] - logsumexp_v logits[t][v]
 *   kl_t   = exp(d) - d - 1 with d = ref_logp[t] - logp_t  (when ref_logp is given):
 *            the per-token KL estimate of the policy from the reference, >= 0 and zero
 *            exactly where the two agree (the pages fix no KL form; their 2M-token runs
 *            used beta = 0).
 * logits: [T][V] dtype (bf16 or fp32), targets: int32 [T], ref_logp: fp32 [T] or NULL;
 * outputs fp32 [T]: logp_out (required), lse_out (natural-log logsumexp, optional),
 * kl_out (optional, requires ref_logp).  Each row is read once.  No workspace.
 * Errors: LS_ERR_INVALID_ARG for a bad dtype, T < 0, V <= 0, a missing or unaligned
 * required pointer, or kl_out without ref_logp; a target outside [0, V) records
 * LS_ERR_DEVICE_CHECK (see ls_last_device_error) and yields NaN for that token. */
ls_status ls_grpo_logp(const void* logits, ls_dtype dtype, int64_t T, int V,
                       const int32_t* targets, const float* ref_logp, float* logp_out,
                       float* lse_out, float* kl_out, ls_stream_t stream);

/* ---------------------------------------------------------------- Gated-DeltaNet replay
 * The hybrid model's Gated-DeltaNet layers keep only the compact recurrent state at the
 * end of the prompt, and each response is replayed from it with that state stopgrad
 * (digest, "Method" step 1 and "Qwen implementation"; explainer, "Two incompatible
 * architectures", Qwen bullet).  The pages give no equations for the layer; the
 * recurrence is the gated delta rule (Yang, Kautz & Hatamizadeh, "Gated Delta Networks:
 * Improving Mamba2 with Delta Rule", ICLR 2025), per head h and response token t:
 *   S_t = exp(g_t) S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,   S_0 = state0[h]
 *   o_t = S_t (scale q_t)
 * S is a 128 x 128 fp32 matrix (d_v x d_k, row-major).  Heads are independent; for
 * grouped key heads the caller passes each value head's q and k.
 *   state0     fp32 [H][128][128]: the captured state (read only)
 *   q, k, v    bf16 [R][H][128]; k is used as given (the layer normalises it)
 *   g, beta    fp32 [R][H]: log of the decay (g <= 0 in the layer) and the write strength
 *   o          bf16 [R][H][128]
 *   state_out  fp32 [H][128][128] or NULL: the state after the last token (running the
 *              prompt from a zero state with state_out set is the capture)
 * Work is done in 64-token chunks; the result does not depend on R's split into chunks
 * beyond rounding.  R == 0 copies state0 to state_out.  workspace: the *_workspace
 * query's bytes (about 0.33 MB (forward) / 0.6 MB (backward) per head and 64 tokens).
 * Errors as for the attention calls; LS_ERR_UNSUPPORTED when ceil(R / 64) * H > 65535. */
ls_status ls_gdn_replay_fwd_workspace(int R, int H, size_t* bytes);
ls_status ls_gdn_replay_fwd(const float* state0, const void* q, const void* k, const void* v,
                            const float* g, const float* beta, int R, int H, float scale, void* o,
                            float* state_out, void* workspace, size_t workspace_bytes,
                            ls_stream_t stream);

/* ls_gdn_replay_bwd: gradients of the replayed response with the captured state
 * stopgrad (the gradient that would reach state0 is dropped).  d_o: bf16 [R][H][128];
 * dq, dk, dv: fp32 [R][H][128]; dg, dbeta: fp32 [R][H]; accumulate != 0 adds into them.
 * The forward's chunk quantities are recomputed; inputs as for the forward. */
ls_status ls_gdn_replay_bwd_workspace(int R, int H, size_t* bytes);
ls_status ls_gdn_replay_bwd(const float* state0, const void* q, const void* k, const void* v,
                            const float* g, const float* beta, const void* d_o, int R, int H,
                            float scale, int accumulate, float* dq, float* dk, float* dv, float* dg,
                            float* dbeta, void* workspace, size_t workspace_bytes,
                            ls_stream_t stream);

/* ---------------------------------------------------------------- latent (MLA) replay
 * The GLM path keeps its multi-head latent attention state as latent pages held in CPU
 * memory and replays each response over them (explainer, "Two incompatible
 * architectures, same transaction", GLM bullet).  The pages give no equations for the
 * layer; it is multi-head latent attention (DeepSeek-V2, 2024) with the key
 * up-projection absorbed into the query.  Every position j keeps one row shared by all
 * heads, its latent c_j (512 values) followed by its rotary key r_j (64 values); the
 * caller passes each head's absorbed query (576 values), and
 *   s_{t,h,j} = softmax_scale * <q_{t,h}, [c_j ; r_j]>,  j over all P prompt rows and
 *               the response rows j <= t
 *   lse_{t,h} = log sum_j exp(s_{t,h,j})        (natural log)
 *   o_{t,h}   = sum_j exp(s_{t,h,j} - lse_{t,h}) c_j   (512 values)
 * The value up-projection and the output projection are weights (the caller's).
 *
 * ls_latent_cache: the captured prompt rows of one latent-attention layer.
 *   pool        bf16 [num_pages][page_size][576]; may be pinned host memory that the
 *               GPU reads directly (on a Grace-Blackwell node, Grace memory behind
 *               NVLink-C2C): capture writes it there and the replay reads it there.
 *   page_table  int32 [num_logical_pages] in GPU memory: logical page -> physical page.
 *   num_tokens  P <= num_logical_pages * page_size.
 * Supported: page_size a power of two in [32, 4096]; num_pages * page_size < 2^31.
 *
 * ls_capture_latent: pool[pt[p / ps]][p % ps][:] = lat[p - start_pos][:] for p in
 * [start_pos, start_pos + n); lat bf16 [n][576].  Bit copy; a page id outside the pool
 * skips the row and sets LS_ERR_DEVICE_CHECK.
 *
 * ls_mla_replay_fwd: the forward of one response of R tokens with H heads.
 * q: bf16 [R][H][576]; lat_resp: bf16 [R][576] (the response's own rows); o: bf16
 * [R][H][512]; lse: fp32 [R][H].  num_splits (>= 1) cuts the prompt into that many
 * ranges of 64-row tiles, merged by log-sum-exp; the result does not depend on it
 * beyond rounding.  softmax_scale finite and > 0.  R == 0 is a no-op; P == 0 is causal
 * attention over the response rows.  Inputs must be finite (a row past a query's
 * causal bound has weight zero, and zero times a non-finite value is not zero).
 * LS_ERR_UNSUPPORTED when R x H >= 2^31.
 *
 * ls_mla_replay_bwd: the backward of ls_mla_replay_fwd with the prompt rows stopgrad
 * (LongStraw paper digest, Method, last paragraph: the captured state takes no
 * gradient).  With P = exp(s - lse), D_{t,h} = <dO_{t,h}, o_{t,h}>, dP_j = <dO, c_j> and
 * dS = P (dP - D):
 *   dq_{t,h} = softmax_scale sum_j dS_{t,h,j} [c_j ; r_j]     (all visible rows j)
 *   dlat_j   = sum_{t >= j} sum_h ( P_{t,h,j} [dO_{t,h} ; 0] + softmax_scale dS_{t,h,j} q_{t,h} )
 * for the response's own rows j (the latent is both key and value; its rotary part is a
 * key only).  q, lat_resp, R, H, softmax_scale and the cache as for the forward; o
 * (bf16 [R][H][512]) and lse (fp32 [R][H]) are the forward's outputs, d_o bf16
 * [R][H][512].  dq: fp32 [R][H][576]; dlat: fp32 [R][576]; both overwritten.
 * num_splits (>= 1) cuts the prompt into ranges of 32-row tiles whose partial dq are
 * added in a fixed order (the result does not depend on it beyond rounding; a given
 * split count gives the same bits every call).  Workspace from
 * ls_mla_replay_bwd_workspace (never zero for R > 0).  R == 0 is a no-op. */
typedef struct {
  void* pool;
  const int32_t* page_table;
  int32_t num_pages;
  int32_t num_logical_pages;
  int32_t page_size;
  int64_t num_tokens;
} ls_latent_cache;

ls_status ls_capture_latent(const ls_latent_cache* cache, const void* lat, int64_t start_pos,
                            int64_t n, ls_stream_t stream);
ls_status ls_mla_replay_fwd_workspace(const ls_latent_cache* cache, int R, int H, int num_splits,
                                      size_t* bytes);
ls_status ls_mla_replay_fwd(const ls_latent_cache* cache, const void* q, const void* lat_resp,
                            int R, int H, float softmax_scale, int num_splits, void* o,
                            float* lse, void* workspace, size_t workspace_bytes,
                            ls_stream_t stream);
ls_status ls_mla_replay_bwd_workspace(const ls_latent_cache* cache, int R, int H, int num_splits,
                                      size_t* bytes);
ls_status ls_mla_replay_bwd(const ls_latent_cache* cache, const void* q, const void* lat_resp,
                            const void* o, const float* lse, const void* d_o, int R, int H,
                            float softmax_scale, int num_splits, float* dq, float* dlat,
                            void* workspace, size_t workspace_bytes, ls_stream_t stream);

/* ---------------------------------------------------------------- query / key stage
 * What a layer does to its projections before attention: the RMS norm of every query and
 * key head and the rotary positions, in one pass, at the layouts the projections have
 * and the replay calls want.  The pages begin at queries and keys as attention takes them and
 * say nothing of this stage, so the common formula is taken.  For a head x of 128 values at
 * token t:
 *   r = 1 / sqrt(mean_i x_i^2 + eps),   u_i = x_i r (w_offset + w_i),
 *   y = u, with each pair (a, b) of its first rot_dim values turned by the pair's angle
 *       p inv_freq[j]: (a cos - b sin, b cos + a sin), p = positions[pair_axis[j]][t].
 * Everything is computed in fp32 and rounded to bf16 once.  The angle's part of a turn is
 * a 64-bit fixed-point number, off by at most 2^-54 of a turn per position (2^-32 at position
 * 4,194,304) for frequencies up to 2 pi however many turns it passes; it is rounded to fp32,
 * by at most 2^-26 of a turn, where its cosine and sine are taken.  A row takes only its own
 * values: a non-finite one reaches no other row.
 *
 * ls_qkv_view: rows of 128 values at q + t q_stride[0] + h q_stride[1] elements (k and v
 * alike), so that a packed projection's slices need no copy.  Strides are multiples of 8
 * elements; rows of an output may not overlap.  An output may be the input itself (the
 * same pointers and strides), otherwise the two may not overlap.
 * ls_qk_norm: weights [128] of type w_dtype, or NULL for none (u_i = x_i r whatever
 * w_offset is); w_offset is 1 for weights that are stored around zero.  A NULL ls_qk_norm* leaves the norm out (y = the turned x).
 * ls_rotary: rot_dim a multiple of 16 up to 128 (0, or a NULL ls_rotary*: no rotation);
 * inv_freq fp64 [rot_dim / 2] (finite), radians per position; pair_axis int32 [rot_dim / 2]
 * gives the axis of each pair (time, height, width, ... of image and video tokens), NULL
 * with one axis; pairs are (j, j + rot_dim / 2), or (2 j, 2 j + 1) when interleaved.
 * positions int32 [axes][T], any sign.  An axis outside [0, axes) sets
 * LS_ERR_DEVICE_CHECK and is taken as axis 0. */
typedef struct {
  void* q;
  void* k;
  void* v;
  int64_t q_stride[2]; /* token, head (elements) */
  int64_t k_stride[2];
  int64_t v_stride[2];
} ls_qkv_view;

typedef struct {
  const void* wq;
  const void* wk;
  ls_dtype w_dtype;
  float w_offset;
  float eps; /* > 0, a normal number, at most 3e38 */
} ls_qk_norm;

typedef struct {
  const double* inv_freq;
  const int32_t* pair_axis;
  int32_t rot_dim;
  int32_t axes; /* 1 to 8 */
  int32_t interleaved;
} ls_rotary;

/* The K and V pages of one layer, as in ls_kv_cache:
 * bf16 [num_pages][num_kv_heads][page_size][128]. */
typedef struct {
  void* k_pool;
  void* v_pool;
  int32_t num_pages;
  int32_t page_size;
  int32_t num_kv_heads;
  int32_t head_dim;
} ls_page_pool;

/* Forward: out.q, out.k from x.q, x.k; v (when x.v is given) is copied to out.v.  All bf16.
 * T == 0 is a no-op. */
ls_status ls_qk_norm_rope_fwd(const ls_qkv_view* x, int64_t T, int Hq, int Hkv,
                              const ls_qk_norm* norm, const ls_rotary* rotary,
                              const int32_t* positions, const ls_qkv_view* out,
                              ls_stream_t stream);

/* The forward with keys and values written into pages instead (a chunk of the prompt on
 * its way into the cache, or the new tokens of a decode step): token t's key and value
 * heads go to slot slots[t] = page * page_size + offset; out.q as above (out.k, out.v are
 * not used).  slots[t] < 0 marks a padding token: nothing of it is written.  A slot
 * outside the pool sets LS_ERR_DEVICE_CHECK and writes no key or value.  Two tokens may
 * not share a slot (either may stay). */
ls_status ls_qk_norm_rope_append(const ls_page_pool* pool, const ls_qkv_view* x, int64_t T,
                                 int Hq, const ls_qk_norm* norm, const ls_rotary* rotary,
                                 const int32_t* positions, const int32_t* slots,
                                 const ls_qkv_view* q_out, ls_stream_t stream);

/* Backward.  x: the forward's inputs (x.v is not read; without a norm nothing of x is).
 * dy: gradients of its outputs, of type dy_dtype (the replay backward's dq, dk_resp and
 * dv_resp are fp32); dx: bf16 gradients of its inputs, dx.v (when dy.v is given) the
 * rounded dy.v.  dwq, dwk: fp32 [128] weight gradients, each or both NULL when not wanted;
 * accumulate != 0 adds into them.  With g = dy turned back, xh = x r, h = g (w_offset + w):
 *   dx = r (h - xh mean_i(h_i xh_i)),   dw_i = sum over tokens and heads of g_i xh_i.
 * dw is summed in fp32 in a fixed order (by rows of a block, then by blocks).  dx may be x
 * itself (same pointers and strides).  workspace: the query's bytes, needed for dwq or dwk
 * only.  T == 0 leaves dx alone and gives (or adds) zero weight gradients. */
ls_status ls_qk_norm_rope_bwd_workspace(int64_t T, size_t* bytes);
ls_status ls_qk_norm_rope_bwd(const ls_qkv_view* x, int64_t T, int Hq, int Hkv,
                              const ls_qk_norm* norm, const ls_rotary* rotary,
                              const int32_t* positions, const ls_qkv_view* dy,
                              ls_dtype dy_dtype, int accumulate, const ls_qkv_view* dx,
                              float* dwq, float* dwk, void* workspace, size_t workspace_bytes,
                              ls_stream_t stream);

/* ---------------------------------------------------------------- growing responses
 * ls_extend_pages: make room for new tokens of `members` sequences whose pages come from
 * one pool, and say where they go; lengths and counts stay on the device, so a captured
 * graph can run it step after step.  Member m holds lens[m] tokens in the pages of row m
 * of block_table (int32 [members][max_blocks], logical -> physical page) and receives
 * add[m] more.  The pages still missing, ceil((len + add) / page_size) -
 * ceil(len / page_size), are taken in member order from free_list[*used], free_list[*used
 * + 1], ... and entered into the table; other entries are left as they are.
 *   slots      int32 [capacity]: page * page_size + offset of every new token, members one
 *              after the other; -1 behind the last token
 *   positions  int32 [axes][capacity] or NULL: pos0 + index within the response (the
 *              same on every axis), 0 behind the last token
 *   lens_out   int32 [members]: lens + add;  used_out int32 [1]: *used + pages taken.
 *              Each may be the input itself (in place), and lens_out may be add.
 *              Other arrays may not overlap.  Without members lens, add and lens_out may be
 *              NULL.
 * A member out of use has lens[m] < 0 and add[m] == 0 and is passed over.  All or nothing:
 * when an add is negative, a member out of use grows, a row of the table is full, the
 * free list ends or the tokens exceed capacity, LS_ERR_DEVICE_CHECK is recorded, every
 * slot is -1, every position 0, and lens_out and used_out repeat the inputs.  A page id
 * outside [0, num_pages) sets LS_ERR_DEVICE_CHECK and gives slot -1.  members <= 1024;
 * page_size a power of two in [16, 4096]; slots and positions 16-byte aligned, the other
 * arrays 4-byte. */
ls_status ls_extend_pages(int32_t* block_table, int members, int max_blocks, int page_size,
                          int num_pages, const int32_t* lens, const int32_t* add,
                          const int32_t* free_list, int num_free, const int32_t* used, int pos0,
                          int axes, int64_t capacity, int32_t* slots, int32_t* positions,
                          int32_t* lens_out, int32_t* used_out, ls_stream_t stream);

/* The same for a step that has `rows` rows of every member, whoever adds how many (members
 * that have ended add none): slots is int32 [members][rows], positions [axes][members][rows],
 * and member m's add[m] new tokens are the last of its rows; slot -1 and position 0 before
 * them.  So row r of member m is its (rows - r)-th newest token, as ls_decode_attn with
 * n = rows takes it.  An add above rows is refused like the others.  (Packed, a member that
 * adds nothing moves every later member's tokens up.)
 *
 * ls_extend_drafts: the same for a step of drafted tokens (ls_draft_tree below).  add may be NULL:
 * all rows of every member in use.  added int32 [members], no other array: what member m got,
 * add[m] or, from a refused call, 0; as the `drafted` of the step's other calls it makes a step
 * without room one that changes nothing. */
ls_status ls_extend_pages_by_member(int32_t* block_table, int members, int max_blocks,
                                    int page_size, int num_pages, const int32_t* lens,
                                    const int32_t* add, const int32_t* free_list, int num_free,
                                    const int32_t* used, int pos0, int axes, int rows,
                                    int32_t* slots, int32_t* positions, int32_t* lens_out,
                                    int32_t* used_out, ls_stream_t stream);
ls_status ls_extend_drafts(int32_t* block_table, int members, int max_blocks, int page_size,
                           int num_pages, const int32_t* lens, const int32_t* add,
                           const int32_t* free_list, int num_free, const int32_t* used, int pos0,
                           int axes, int rows, int32_t* slots, int32_t* positions,
                           int32_t* lens_out, int32_t* used_out, int32_t* added,
                           ls_stream_t stream);

/* The responses of a group in their own pages: member m's key j lies in page
 * block_table[m][j / page_size] of `pool`; lens int32 [members] on the device, negative
 * for a member out of use.  Entries behind a member's length are not read. */
typedef struct {
  ls_page_pool pool;
  const int32_t* block_table; /* int32 [members][max_blocks] */
  const int32_t* lens;
  int32_t members;
  int32_t max_blocks;
} ls_resp_cache;

/* ls_decode_attn: attention of a decode step: the n newest tokens of every member (their
 * keys and values already in its pages, as the last n of its lens[m]) over the shared
 * captured prompt and the member's own response:
 *   s_j = softmax_scale <q_{m,i,h}, k_j>, j over all P prompt positions and the member's
 *         response keys j <= lens[m] - n + i (none when that is negative)
 *   lse = log sum_j exp(s_j) (natural log),  o = sum_j exp(s_j - lse) v_j
 * Each prompt K/V tile is read once for all members.  q, o: bf16 [members][n][Hq][128];
 * lse: fp32 [members][n][Hq].  A token that sees no key at all (P == 0 and an empty
 * response) gets o = 0 and lse = -inf; the rows of a member out of use are not written.
 * A member's result takes its own queries and keys and the prompt only.  Values must be
 * finite where a row may not look (a later new token's value times zero weight); what
 * lies behind a sequence's end in its last page may be anything.  A length past
 * max_blocks * page_size is cut there and sets LS_ERR_DEVICE_CHECK, as does a page id
 * outside its pool (its keys and values count as zeros).  n * Hq / num_kv_heads <= 128,
 * members <= 1024, and members * n * Hq / num_kv_heads rows of at most 128 per SM, else
 * LS_ERR_UNSUPPORTED.  Two launches; the lengths may change between replays
 * of a captured graph, the pointers and P may not.  members == 0 is a no-op. */
ls_status ls_decode_attn_workspace(const ls_kv_cache* cache, const ls_resp_cache* resp, int n,
                                   int Hq, size_t* bytes);
ls_status ls_decode_attn(const ls_kv_cache* cache, const ls_resp_cache* resp, const void* q,
                         int n, int Hq, float softmax_scale, void* o, float* lse,
                         void* workspace, size_t workspace_bytes, ls_stream_t stream);

/* ---------------------------------------------------------------- drafted trees
 * A decode step over drafted tokens: every member's draft is a tree of tokens that the policy
 * looks at in one pass; of it the path that the policy itself chooses is kept.  (The pages
 * describe no rollout; this is the decode step above for several continuations at once.)
 *
 * A step has n rows a member (1 to 128), and the last drafted[m] of them are its draft; drafted
 * NULL: all n.  The rows before are padding.  lens[m] counts the draft, whose keys are the
 * member's last ones: row r's is key lens[m] - n + r, and keys before lens[m] - drafted[m] are
 * the context.  (ls_extend_pages_by_member with rows = n and add = drafted gives these slots.)
 * parents int32 [members][n]: row r's node continues node parents[m][r], an earlier row of the
 * draft, or -1: the context.  Another value sets LS_ERR_DEVICE_CHECK and is taken as -1, as does
 * a drafted[m] outside 0 .. min(n, lens[m]), which is cut.  A member out of use (lens[m] < 0)
 * has no draft.  members <= 1024.
 *
 * ls_draft_tree: the plan of a step, once for all layers.
 *   visible    int32 [members][n][ceil(n / 32)]: bit j of row r (bit j % 32 of word j / 32) is
 *              set when r sees row j: itself and its ancestors.  0 in padding rows
 *   positions  int32 [axes][members][n] or NULL: pos0 + context + depth (a node behind the
 *              context has depth 0), the same on every axis; 0 in padding rows */
ls_status ls_draft_tree(const int32_t* parents, const int32_t* lens, const int32_t* drafted,
                        int members, int n, int pos0, int axes, int32_t* visible,
                        int32_t* positions, ls_stream_t stream);

/* ls_decode_attn_tree: ls_decode_attn for trees.  Row r of member m sees all P prompt
 * positions, the member's context, and of its draft the rows whose bits are set in
 * visible[m][r] (any bits, not only a tree's; bits of padding rows and behind n count for
 * nothing).  q, o, lse as there; padding rows of o and lse are not written, nor are those of a
 * member out of use; a row that sees no key gets o = 0 and lse = -inf.  resp->lens counts the
 * drafts.  n <= 128, Hq / num_kv_heads <= 128, and members * n * Hq / num_kv_heads rows of at
 * most 128 per SM, else LS_ERR_UNSUPPORTED.  Values must be finite where a row may not look
 * within the draft.  The rest as ls_decode_attn. */
ls_status ls_decode_attn_tree_workspace(const ls_kv_cache* cache, const ls_resp_cache* resp, int n,
                                        int Hq, size_t* bytes);
ls_status ls_decode_attn_tree(const ls_kv_cache* cache, const ls_resp_cache* resp, const void* q,
                              int n, int Hq, const int32_t* visible, const int32_t* drafted,
                              float softmax_scale, void* o, float* lse, void* workspace,
                              size_t workspace_bytes, ls_stream_t stream);

/* ls_accept_draft: which nodes the policy keeps.  tokens int32 [members][n]: the drafted tokens;
 * chosen int32 [members][n]: the policy's own token behind each row (sampled or the most likely
 * one: the caller's).  The draft's first row is always kept (its token is the one chosen in the
 * step before); then, from a kept row, its child whose token is the one chosen there (the first
 * such row; negative tokens match nothing), and so on.  Other rows with parent -1 are not kept.
 *   rows    int32 [members][n]: the kept rows, ascending; -1 behind them
 *   count   int32 [members]: how many;  ends int32 [members]: context + count (a negative
 *           length as it is)
 *   follow  int32 [members]: the token chosen behind the last kept row; -1 without a draft */
ls_status ls_accept_draft(const int32_t* parents, const int32_t* tokens, const int32_t* chosen,
                          const int32_t* lens, const int32_t* drafted, int members, int n,
                          int32_t* rows, int32_t* count, int32_t* follow, int32_t* ends,
                          ls_stream_t stream);

/* ls_compact_rows: in the pages of every layer, the key and value of rows[m][i] become the
 * i-th of those behind member m's context.  Layer l's pools begin l * layer_stride values (a
 * multiple of 8, at least a pool's size) behind pool's.  rows, count as from ls_accept_draft
 * (rows ascending within the draft; a count or row that is not sets LS_ERR_DEVICE_CHECK and moves
 * nothing of the member, as does a length past the table; a page id outside the pool sets it and
 * moves nothing of the row).  Lengths are not changed: ls_trim_pages to `ends` follows.  No two
 * members may hold a page of their drafts together. */
ls_status ls_compact_rows(const ls_page_pool* pool, int layers, int64_t layer_stride,
                          const int32_t* block_table, int max_blocks, const int32_t* lens,
                          const int32_t* drafted, int members, int n, const int32_t* rows,
                          const int32_t* count, ls_stream_t stream);

/* ---------------------------------------------------------------- pages given back and shared
 * Beside ls_extend_pages, on the same arrays.  shared int32 [num_pages]: how many members hold
 * a page besides the first (0 for pages that ls_extend_pages gives out).
 *
 * ls_trim_pages: member m keeps its first new_lens[m] <= lens[m] tokens; new_lens[m] < 0 puts
 * it out of use (lens -1).  Pages behind the new end lose m as an owner, and those without one
 * left go back: they become free_list[used - freed .. used), in member and block order, and
 * used falls by their number.  The table's entries stay as they are.  shared NULL: no page has
 * a second owner.  lens_out and used_out may be the inputs themselves (lens_out also new_lens).
 * All or nothing: when a new length passes the old one (a member out of use has a negative
 * one), a length its row of the table, a page id the pool, a page is given back more often than
 * it is held, more pages than are in use, or a member would end inside a page that others
 * still hold (it would write there next; branch it with ls_fork_pages instead),
 * LS_ERR_DEVICE_CHECK is recorded, lens_out and used_out repeat the inputs, and nothing else
 * changes. */
ls_status ls_trim_pages(const int32_t* block_table, int members, int max_blocks, int page_size,
                        int num_pages, const int32_t* lens, const int32_t* new_lens,
                        int32_t* free_list, int num_free, const int32_t* used, int32_t* shared,
                        int32_t* lens_out, int32_t* used_out, ls_stream_t stream);

/* ls_fork_pages: member m with src[m] >= 0 becomes a branch of member src[m]: its first keep[m]
 * tokens (keep NULL: all).  m is out of use or holds no tokens, src[m] is in use and no branch
 * of this call.  Whole pages are shared; for a partial last one m takes a page of its own, in
 * member order from free_list[*used] on, into which its rows are to be copied, in every layer:
 *   copies  int32 [3][members]: from page, to page, rows; (-1, -1, 0) where there is none.
 *           The three rows are ls_copy_pages' from, to and rows
 * All or nothing, as ls_trim_pages; copies then says that there is none.  src[m] < 0: m stays
 * as it is.  lens_out and used_out may be the inputs themselves. */
ls_status ls_fork_pages(int32_t* block_table, int members, int max_blocks, int page_size,
                        int num_pages, const int32_t* lens, const int32_t* src, const int32_t* keep,
                        const int32_t* free_list, int num_free, const int32_t* used,
                        int32_t* shared, int32_t* copies, int32_t* lens_out, int32_t* used_out,
                        ls_stream_t stream);

/* ls_copy_pages: the first rows[i] rows (rows NULL: all) of every KV head of page from[i] to
 * page to[i], keys and values, in every layer (as in ls_compact_rows), for i < count.  Bit copy.
 * from[i] and to[i] both negative: nothing.  Another id outside the pool, or rows[i] outside
 * [0, page_size], sets LS_ERR_DEVICE_CHECK and copies nothing of the pair.  A page that is
 * written may appear only once. */
ls_status ls_copy_pages(const ls_page_pool* pool, int layers, int64_t layer_stride, int count,
                        const int32_t* from, const int32_t* to, const int32_t* rows,
                        ls_stream_t stream);

/* ---------------------------------------------------------------- token statistics
 * What rollouts log and objectives are made of, beside the fused loss above.  For a row of
 * logits z, temperature tau (1e-6 to 1e6) and target y:
 *   lse = log sum_v exp(z_v / tau),  logp = z_y / tau - lse,  p_v = exp(z_v / tau - lse),
 *   entropy = -sum_v p_v log p_v,
 *   alternatives: the top (0 to 32, <= V) largest z_v / tau - lse with their ids, equal ones by
 *   the lowest id first.
 * logits: T rows of V values of type dtype, row_stride >= V values apart (a padded vocabulary's
 * rows need no copy; values behind V are not read), aligned to their own size.  targets int32
 * [T]: -1 marks a padding row, whose outputs are 0 and ids -1 and whose logits are not read;
 * another one outside [0, V) sets LS_ERR_DEVICE_CHECK and gives logp = NaN.  Outputs fp32 [T],
 * each or NULL: logp (needs targets), lse, entropy; targets NULL: no row is padding.  top_logp
 * fp32 and top_ids int32 [T][top] (4-byte aligned, as every array here).  A logit of -inf has
 * probability 0, as has one of the type's lowest value beside ordinary ones (a row of such values
 * alone is as probable as their distances say).  A row with a NaN or +inf, or without a finite
 * logit, has NaN numbers, but for the lse of a row of -inf, which is -inf; its ids are of V or -1.
 *
 * Backward, with upstream d_logp [T], d_entropy [T] (each or NULL) and d_top [T][top] (top 0:
 * none) and G = d_logp + sum_j d_top_j:
 *   dlogits_v = (d_logp 1[v = y] + sum_j d_top_j 1[v = top_ids_j]
 *                - p_v (G + d_entropy (log p_v + entropy))) / tau
 * of type dtype, rows d_row_stride >= V apart (values behind V are left alone); zeros in padding
 * rows.  It may be the logits themselves (same pointer and stride), otherwise the two may not
 * overlap.  lse and entropy (needed with d_entropy) are the forward's, top_ids any ids.  p_v is
 * that of the lse given: the rounding of lse to fp32 (2^-24 |lse| at most) is a relative error of
 * p_v.  That is 1/500 for a logit of 30 at a temperature of 1e-3 and all of p_v at 1e-6:
 * temperatures below 1e-3 are LS_ERR_UNSUPPORTED.  A target or id outside [0, V) sets LS_ERR_DEVICE_CHECK and makes its row
 * NaN. */
ls_status ls_token_logp_fwd_workspace(ls_dtype dtype, int64_t T, int V, int top, size_t* bytes);
ls_status ls_token_logp_fwd(const void* logits, ls_dtype dtype, int64_t T, int V, int64_t row_stride,
                            const int32_t* targets, float temperature, int top, float* logp,
                            float* lse, float* entropy, float* top_logp, int32_t* top_ids,
                            void* workspace, size_t workspace_bytes, ls_stream_t stream);
ls_status ls_token_logp_bwd(const void* logits, ls_dtype dtype, int64_t T, int V, int64_t row_stride,
                            const int32_t* targets, float temperature, const float* lse,
                            const float* entropy, int top, const int32_t* top_ids,
                            const float* d_logp, const float* d_entropy, const float* d_top,
                            void* dlogits, int64_t d_row_stride, ls_stream_t stream);

/* ---------------------------------------------------------------- checks
 * ls_validate_page_table: enqueue a check that every entry of the page table covering
 * the cache's num_tokens lies in [0, num_pages) and that no physical page is used
 * twice; a failure sets LS_ERR_DEVICE_CHECK in the device error word.
 * ls_last_device_error: synchronise `stream`, return the first device-side error
 * recorded on the current device since the last call (LS_OK if none) and clear it. */
ls_status ls_validate_page_table(const ls_kv_cache* cache, void* workspace,
                                 size_t workspace_bytes, ls_stream_t stream);
ls_status ls_validate_page_table_workspace(const ls_kv_cache* cache, size_t* bytes);
ls_status ls_last_device_error(ls_stream_t stream);

const char* ls_status_string(ls_status status);

/* Diagnostic: number of kernel launches this library has issued in the process (all
 * devices), e.g. to count the launches of one step. */
uint64_t ls_kernel_launches(void);

/* Diagnostic (the pages have no counterpart): enqueue one block that waits, through the
 * pipelines' own bounded mbarrier wait, on a barrier nothing completes.  After the
 * wait's time limit (about 2 s of SM clock) the block records LS_ERR_TIMEOUT in the
 * device error word and exits, so a following ls_last_device_error() returns
 * LS_ERR_TIMEOUT and the context stays usable.  Returns LS_OK once enqueued,
 * LS_ERR_CUDA if the launch fails.  Used by the tests of the failure path. */
ls_status ls_selftest_wait_timeout(ls_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* LONGSTRAW_H */
