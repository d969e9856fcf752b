/*
 * g4attn.h -- C ABI of the GB300 (sm_103a) Gemma-4 E-series dual-geometry
 * attention path.
 *
 * The path, per layer of an attention-only stack:
 *   1. g4_kv_append_normrope: per-head RMSNorm of q and k (plain x-hat * w,
 *      eps inside the mean), weight-less RMSNorm of v, rotate_half RoPE on q
 *      and k, and the write of k and v into the layer's KV cache.
 *   2. g4_attn_prefill / g4_attn_decode: causal GQA softmax attention with
 *      score scale attn_scale (1.0 for Gemma-4), windowed on sliding layers,
 *      over the cache of the layer itself or, on a shared-KV tail layer, of
 *      its source layer.  g4_attn_encoder: the bidirectional (encoder) form.
 *
 * Sources (page title + item):
 *   cortiq-engine g4e.rs: `rms`, `rms_plain`, `G4eGlobals` (inv_freq tables,
 *     window counted with the current token), `G4eLayer` (kv_share_src,
 *     sliding, hd),
 *     `g4e_forward` attention block.
 *   ferrox-models gemma4_engine.rs: `Gemma4Hparams` (head_dim per type,
 *     has_kv, kv_reuse_layer, rope_theta_for, attention_scale = 1.0),
 *     `forward_token_on_worker` (norm per head, RoPE, push, windowed /
 *     unwindowed causal GQA attention, shared-KV head_dim check).
 *   taconite-embeddinggemma2 model.rs: `rope_half`, `text_attention`
 *     (rotate_half pairing, head grouping kh = hh / group).
 *   turbospark-runtime gemma4/attn.rs: `encode_gemma4_layer_attn_and_router`
 *     (RMS_EPS = 1e-6, rotated_pairs, kv_start = seq_len - sliding_window).
 *
 * Conventions shared by every entry point
 *   - All tensor arguments are DEVICE pointers owned by the caller; the
 *     library allocates no device memory and keeps no state between calls
 *     except a thread-local error message, one device-side error word (see
 *     g4_take_device_error), the built-in scratch of g4_attn_decode_noalloc
 *     and 64 pairs of work-item counters of the bf16 prefill (see
 *     g4_attn_prefill), the last three static device variables; and on the
 *     host, per thread, the RoPE frequencies of the last four (theta, head_dim,
 *     rotated pairs) met, and per device its kernels' launch attributes.
 *   - Every call is asynchronous on `stream` (a cudaStream_t passed as void*;
 *     NULL is the legacy default stream).  A call that returns G4_OK has only
 *     enqueued work.
 *   - Host-detectable errors return a status before anything is launched;
 *     nothing is written then.  g4_last_error() gives the message.
 *   - Device-side values (positions, lengths) cannot be checked on the host.
 *     Kernels clamp them so that no access leaves the buffers; rows with
 *     out-of-contract values get unspecified contents.
 *   - Pointers to q/k/v/out/cache must be 16-byte aligned.
 *   - dtype is per layer and covers q_in/k_in/v_in, the cache, q_out and the
 *     attention output alike: G4_F32 (float) or G4_BF16 (bfloat16, RNE on
 *     every store).  Norm weights are always float32.  Arithmetic is float32
 *     with float32 accumulation (bf16 tensor-core inputs in bf16 prefill).
 */
#ifndef G4ATTN_H
#define G4ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  G4_OK = 0,
  G4_ERR_INVALID_ARG = 1,    /* null / misaligned pointer, bad size or field      */
  G4_ERR_UNSUPPORTED = 2,    /* head_dim or GQA group not built                    */
  G4_ERR_SHARE_MISMATCH = 3, /* shared layer's source cache has another type,
                                head_dim, kv-head count or dtype                   */
  G4_ERR_CAPACITY = 4,       /* batch or length larger than the cache              */
  G4_ERR_WORKSPACE = 5,      /* decode workspace too small                         */
  G4_ERR_CUDA = 6            /* a CUDA runtime/driver call or launch failed        */
} g4_status;

typedef enum { G4_SLIDING = 0, G4_FULL = 1 } g4_layer_type;
typedef enum { G4_F32 = 0, G4_BF16 = 1 } g4_dtype;

/*
 * Per-layer attention hyperparameters (ferrox-models `Gemma4Hparams`,
 * cortiq-engine `G4eLayer`).
 *   layer_type      G4_SLIDING or G4_FULL.
 *   head_dim        this layer's head width: head_dim on sliding layers,
 *                   global_head_dim on full layers.  64, 128, 256 or 512.
 *   n_heads         query heads H; n_kv_heads Hkv divides it and the group
 *                   H / Hkv is 1, 2, 4 or 8 (with group * head_dim <= 2048).
 *   window          sliding window in tokens, current token included (a key
 *                   j is visible from query i iff j <= i and i - j < window).
 *                   Must be >= 1 on sliding layers; ignored on full layers.
 *   theta           RoPE base (local theta on sliding, model theta on full).
 *   rotary_fraction fraction of the head that is rotated: the first
 *                   floor(head_dim * rotary_fraction / 2) pairs rotate with
 *                   inv_freq[j] = theta^(-2j / head_dim); the other pairs have
 *                   inv_freq 0 (identity).  1.0 on sliding layers, the
 *                   partial-rotary factor (e.g. 0.25) on full layers.
 *   eps             RMSNorm epsilon (1e-6), added to the mean square.
 *   attn_scale      score scale, > 0 (Gemma-4: 1.0).
 *   kv_share_src    -1 if the layer owns its cache, else the index of the
 *                   layer whose cache it reads (see g4_kv_share_src).
 *   dtype           g4_dtype of every tensor of the layer.
 */
typedef struct {
  int32_t layer_type;
  int32_t head_dim;
  int32_t n_heads;
  int32_t n_kv_heads;
  int32_t window;
  float theta;
  float rotary_fraction;
  float eps;
  float attn_scale;
  int32_t kv_share_src;
  int32_t dtype;
} g4_layer_params;

/*
 * One layer's KV cache, caller-owned device memory, layout
 * k[batch][n_kv_heads][max_len][head_dim] (same for v): rows of head_dim
 * contiguous.  Layers that read another layer's cache may leave their entry
 * zeroed.
 *   ring = 0  linear cache: position p lives in row p, positions < max_len.
 *   ring = 1  sliding-window ring buffer (turbospark-runtime gemma4 decode:
 *             `ring_capacity`, `active_ring`): position p lives in row
 *             p mod max_len, any p >= 0, so the cache keeps the last max_len
 *             positions.  Only on a G4_SLIDING cache, with max_len >= the
 *             layer's window (G4_ERR_INVALID_ARG / G4_ERR_CAPACITY otherwise).
 *             A ring of `window` rows serves decode; a prefill chunk of T
 *             tokens needs max_len >= T + window - 1 (see g4_attn_prefill).
 */
typedef struct {
  void* k;
  void* v;
  int32_t layer_type;
  int32_t head_dim;
  int32_t n_kv_heads;
  int32_t max_len;
  int32_t batch;
  int32_t dtype;
  int32_t ring;
} g4_kv_cache;

/*
 * Shared-KV routing (ferrox-models `Gemma4Hparams::kv_reuse_layer`;
 * cortiq-engine g4e.rs module doc).  With first_shared = n_layers - n_shared:
 * returns -1 for layer < first_shared (owns its cache), first_shared - 2 for a
 * sliding tail layer and first_shared - 1 for a full tail layer.
 * is_sliding[n_layers] holds 1 for sliding layers.  Returns -2 on invalid
 * arguments (n_layers < 1, n_shared outside [0, n_layers), layer out of range,
 * NULL is_sliding, or a source index < 0).  Host only.
 */
int32_t g4_kv_share_src(int32_t n_layers, int32_t n_shared, const int32_t* is_sliding, int32_t layer);

/*
 * Step a4: fused norm -> RoPE -> KV append for B*T tokens of one layer.
 *   q_in       [B][T][n_heads][head_dim]      raw q projections
 *   k_in, v_in [B][T][n_kv_heads][head_dim]   raw k / v projections; must be
 *              NULL on a shared layer (kv_share_src >= 0), non-NULL otherwise.
 *              A full layer whose v projection is its k projection
 *              (turbospark-runtime gemma4 `attention_k_eq_v`) passes the raw
 *              k as v_in too; v is then the weight-less norm of the raw k.
 *   q_norm_w   [head_dim] float32 weight shared by all q heads
 *   k_norm_w   [head_dim] float32 weight shared by all k heads (NULL on a
 *              shared layer).  v has no weight.
 *   positions  [B][T] int32: the RoPE position of each token and the cache row
 *              it is written to (row = position on a linear cache, position
 *              mod max_len on a ring).  Negative positions, and positions
 *              >= max_len of a linear cache, are not written.
 *   q_out      [B][T][n_heads][head_dim] normed + roped q; may equal q_in.
 * The layer's cache is caches[layer] (n_layers entries).  Writes exactly the
 * rows k[b][*][row(positions[b][t])][*] and v[...] for every (b, t); nothing
 * else in the cache changes.  Two tokens of one call that map to the same
 * ring row leave either one there.  RoPE angles are pos * inv_freq[j] with
 * inv_freq held in float32 and the angle reduced in float64.
 */
g4_status g4_kv_append_normrope(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                                int32_t layer, const void* q_in, const void* k_in, const void* v_in,
                                const float* q_norm_w, const float* k_norm_w, const int32_t* positions,
                                int32_t B, int32_t T, void* q_out, void* stream);

/*
 * Step a5 (+ a7): prefill attention of T new tokens per sequence.
 *   q            [B][T][n_heads][head_dim], normed + roped (g4_kv_append_normrope's q_out)
 *   q_start_pos  [B] int32 device: token t of sequence b sits at position
 *                q_start_pos[b] + t; the cache of the source layer must
 *                already hold positions [0, q_start_pos[b] + T).  On a ring
 *                cache those are the last max_len of them, and every key the
 *                chunk needs is still there when max_len >= T + window - 1
 *                (checked: G4_ERR_CAPACITY); a bf16 ring also needs max_len
 *                a multiple of 128, the key tile (G4_ERR_UNSUPPORTED).
 *   out          [B][T][n_heads][head_dim]
 * Reads caches[src], src = kv_share_src < 0 ? layer : kv_share_src, which must
 * match the layer's type, head_dim, n_kv_heads and dtype
 * (G4_ERR_SHARE_MISMATCH otherwise).  bf16 runs on the tcgen05 tensor cores
 * (bf16 operands, float32 accumulation, P rounded to bf16); f32 runs on CUDA
 * cores in float32.  The bf16 kernel is persistent: its CTAs draw work items
 * from a counter pair the library keeps in device memory, one of 64 taken in
 * turn per call and cleared by the launch when it ends; so at most 64 bf16
 * prefill launches may be in flight at the same time (any streams).  A CUDA
 * graph keeps the pair it was captured with: replays of one graph, or of two
 * graphs whose prefill captures were a multiple of 64 calls apart, must not
 * overlap.
 */
g4_status g4_attn_prefill(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                          int32_t layer, const void* q, const int32_t* q_start_pos, int32_t B, int32_t T,
                          void* out, void* stream);

/*
 * Bidirectional (encoder) attention, the form of taconite-embeddinggemma2
 * model.rs `text_attention`: no causal mask; a key j is visible from query i
 * iff |i - j| <= window on a sliding layer (the window counts keys on each
 * side, the token itself in the middle), every key on a full layer.
 *   q    [B][T][n_heads][head_dim], normed + roped at positions 0 .. T-1
 *        (g4_kv_append_normrope's q_out with positions[b][t] = t)
 *   out  [B][T][n_heads][head_dim]
 * The keys and values are the same T tokens, rows [0, T) of caches[src]
 * (appended by g4_kv_append_normrope at positions 0 .. T-1; src as in
 * g4_attn_prefill).  A ring cache is refused (G4_ERR_INVALID_ARG); T must
 * not exceed max_len (G4_ERR_CAPACITY).  Score scale attn_scale.  bf16 runs
 * on the tcgen05 tensor cores, f32 on CUDA cores, like g4_attn_prefill (the
 * bf16 kernel takes one of the same 64 work-item counter pairs).
 */
g4_status g4_attn_encoder(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                          int32_t layer, const void* q, int32_t B, int32_t T, void* out, void* stream);

/*
 * Workspace bytes g4_attn_decode / g4_decode_step need for this layer, batch
 * and bound on the sequence lengths (0 means no workspace is needed).
 */
size_t g4_attn_decode_workspace_size(const g4_layer_params* params, int32_t B, int32_t max_seq_len);

/*
 * Step a6 (+ a7): one query token per sequence (decode).
 *   q            [B][n_heads][head_dim], normed + roped
 *   seq_lens     [B] int32 device: keys per sequence INCLUDING the new token,
 *                which sits at position seq_lens[b] - 1 (append it first).
 *                Values are clamped into [1, max_seq_len].
 *   max_seq_len  host-side upper bound of seq_lens, 1..cache max_len (any
 *                value >= 1 on a ring cache); it sizes the split-KV grid and
 *                the workspace.
 *   out          [B][n_heads][head_dim]
 *   workspace    device scratch of at least g4_attn_decode_workspace_size()
 *                bytes (may be NULL when that is 0); caller-owned, 16-byte
 *                aligned.  Zero-fill it once before its first use: it holds
 *                arrival counters that every call leaves at zero again.
 * Sliding layers read keys [max(0, L - window), L), full layers [0, L).  The
 * key range is split across CTAs (split-KV); the CTA that finishes last for a
 * (sequence, kv head) merges the splits with log-sum-exp weights.  Calls
 * sharing a workspace must not overlap on the GPU.
 */
g4_status g4_attn_decode(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                         int32_t layer, const void* q, const int32_t* seq_lens, int32_t B, int32_t max_seq_len,
                         void* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Steps a4 + a6 (+ a7) in one launch: the decode step of one layer from the
 * new token's raw projections.  Same result as g4_kv_append_normrope with
 * positions[b] = seq_lens[b] - 1 (T = 1) followed by g4_attn_decode on its
 * q_out, without the q_out round trip through memory:
 *   q_in         [B][n_heads][head_dim] raw q of the new token
 *   k_in, v_in   [B][n_kv_heads][head_dim] raw k / v (NULL on a shared layer;
 *                the same pointer twice for attention_k_eq_v, as above)
 *   q_norm_w, k_norm_w  float32 [head_dim] (k_norm_w NULL on a shared layer)
 * On a layer that owns its cache the new k / v rows are written to position
 * seq_lens[b] - 1 of caches[layer] (row seq_lens[b] - 1, or that mod max_len
 * on a ring, which overwrites a key the window no longer sees).  Other
 * arguments as g4_attn_decode.
 */
g4_status g4_decode_step(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers, int32_t layer,
                         const void* q_in, const void* k_in, const void* v_in, const float* q_norm_w,
                         const float* k_norm_w, const int32_t* seq_lens, int32_t B, int32_t max_seq_len, void* out,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * The step before the path, fused into it: the q / k / v projections of one
 * layer for B*T tokens, their input RMSNorm, and the per-head norm / RoPE /
 * KV append of g4_kv_append_normrope, on the tcgen05 tensor cores
 * (cortiq-engine g4e.rs `g4e_forward`: `rms(h, attn_norm)`, then `matvec`
 * with wq / wk / wv, then the per-head norm, RoPE and `append`;
 * turbospark-runtime gemma4/attn.rs writes the projections straight into the
 * KV slot and norms / ropes them there).  bf16 only (G4_ERR_UNSUPPORTED for
 * float32 layers).
 *   x        [B][T][D] bf16: the layer input (residual stream), D a multiple
 *            of 64.
 *   w_qkv    [N][D] bf16, N = (n_heads + 2 n_kv_heads) * head_dim rows: the
 *            rows of Wq, then Wk, then Wv (n_heads * head_dim rows, Wq only,
 *            on a shared layer), each column k multiplied by the attention-norm
 *            weight attn_norm_w[k] (folded in once by the caller, as
 *            taconite-embeddinggemma2 model.rs folds RMSNorm weights into its
 *            GEMM operands).  The kernel applies the rest of the input norm,
 *            the row scale (mean(x^2) + eps)^-1/2 with the layer's eps.
 *   q_norm_w, k_norm_w, positions, q_out  as g4_kv_append_normrope (k_norm_w
 *            NULL on a shared layer).
 * q = (x scale) Wq^T etc. accumulate in float32 from bf16 products; the
 * per-head norm, RoPE and the bf16 rounding (to nearest even) follow in
 * float32.  So the stored values are those of g4_kv_append_normrope on the
 * exact projections to within one bf16 unit in the last place, where the
 * float32 accumulation lands next to a rounding boundary.  Writes q_out and
 * the cache rows of the tokens' positions (positions outside a linear cache
 * are not written), nothing else.  The launch takes one 128-token x
 * head_dim output tile per CTA.
 */
g4_status g4_qkv_project_append(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                                int32_t layer, const void* x, int32_t D, const void* w_qkv, const float* q_norm_w,
                                const float* k_norm_w, const int32_t* positions, int32_t B, int32_t T, void* q_out,
                                void* stream);

/*
 * The step after the path: o_proj, the post-attention RMSNorm and the
 * residual add (cortiq-engine g4e.rs `g4e_forward`: `wo`, then the sandwich
 * norm `rms(.., post_attn_norm)` added to the hidden state; ferrox-models
 * gemma4_engine.rs `forward_token_on_worker`: `o_proj`, `post_attn_norm`,
 * residual), on the tcgen05 tensor cores, bf16:
 *   out[m][:] = h[m][:] + rmsnorm(ao[m][:] . w_o^T, post_norm_w, eps)
 *   ao           [M][K] bf16: attention output rows (K = n_heads * head_dim,
 *                a multiple of 64), e.g. g4_attn_prefill's out as [B*T][H*hd]
 *   w_o          [D][K] bf16
 *   post_norm_w  [D] float32; eps added to the mean square
 *   h            [M][D] bf16 residual stream; out [M][D] bf16 (may equal h)
 * D must be a multiple of 256 and at most 2048 (G4_ERR_UNSUPPORTED): the
 * norm's row sum is formed by one thread-block cluster of D / 256 CTAs.
 * Accumulation and the norm in float32; out rounded to nearest even.
 */
g4_status g4_attn_out_residual(const void* ao, int32_t M, int32_t K, const void* w_o, int32_t D,
                               const float* post_norm_w, float eps, const void* h, void* out, void* stream);

/*
 * Bytes of device scratch built into the library for g4_attn_decode_noalloc
 * (8 MiB).  Every GPU that loads the library holds this array until the
 * process exits.
 */
#define G4_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)

/*
 * g4_attn_decode without a workspace argument, for callers that cannot
 * allocate device memory: code that is handed only its input and output
 * buffers (a plugin or custom op inside a host framework that owns every
 * allocation), or a serving loop that must not call cudaMalloc because it
 * synchronises the device and can fail mid-request.  (The pages have no
 * counterpart: this is an interface choice of this library.)
 *
 * Arguments, results and error codes are those of g4_attn_decode; the
 * split-KV partials go to a fixed array of G4_NOALLOC_SCRATCH_BYTES inside
 * the library instead of a caller's workspace.  A call whose split plan
 * (g4_attn_decode_workspace_size) exceeds that size returns
 * G4_ERR_WORKSPACE and launches nothing.  The call allocates nothing.
 *
 * The first call on a device looks up the array's device address (once per
 * device, with that device current); make that first call before any stream
 * capture.  All calls share the one array and it keeps the last call's
 * contents; each call clears the part that must start at zero (the splits'
 * arrival counters, an asynchronous memset on `stream`) once its arguments
 * have passed every check, just before its launch, so a refused call writes
 * nothing.  Calls whose kernels overlap on the GPU (different streams, or
 * several threads) race on the array and must be serialised by the caller.
 */
g4_status g4_attn_decode_noalloc(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                                 int32_t layer, const void* q, const int32_t* seq_lens, int32_t B,
                                 int32_t max_seq_len, void* out, void* stream);

/* ------------------------------------------------------------------------
 * A paged KV cache in 4 bits
 *
 * The cache above is one rectangle of bf16 or float32 rows per layer.  A
 * server that holds many contexts of differing lengths keeps them instead in
 * blocks of 16 to 128 positions, dealt out of a pool as sequences grow, and
 * in 4.5 bits per element, 2 / 0.5625 = 3.6 times fewer bytes than bf16: as much
 * less for decode to stream, and on layers that keep all positions 3.6 times more
 * contexts.  A sequence's blocks hold all its positions on sliding layers too,
 * where the bf16 ring above keeps one window: over a stack that is mostly sliding
 * layers, one table for all of them saves little memory against rings (the
 * 42-layer stack of 20 sliding and 4 full caches: 132 MB per context of 8192
 * positions against 155).  Sliding layers with a table and free list of their own
 * do not need the blocks behind the window: the caller may take such a block away
 * at any time (its entry becomes -1, its id goes onto the free list).
 * (The pages have no counterpart: this is a cache of this library.)
 *
 * What a row holds.  x is the bf16 row that g4_kv_append_normrope would
 * store.  For every 16 consecutive elements, with e = k_exp for k and 0 for v:
 *   s      = RN_e4m3(min(max |x| 2^-e / 6, 448))   one byte
 *   code_d = RN_e2m1(x_d 2^-e / s), 0 where s = 0   four bits
 * (RN: to nearest, ties to even; e2m1 holds 0, 0.5, 1, 1.5, 2, 3, 4, 6 and
 * their negatives and saturates at 6), and the row stands for code_d s 2^e,
 * which bf16 holds exactly.  x is itself correctly rounded, so the bytes are
 * a function of the raw inputs alone, whatever kernel wrote them.  A 16 that
 * holds a NaN or an infinity gets the scale NaN and codes 0, and stands for NaNs.
 *
 * Where it lies.  data[n_blocks][n_kv_heads][block_size / 16] records of
 * 18 head_dim bytes, one per 16 positions of one kv head: K codes (8
 * head_dim bytes), K scales (head_dim), V codes (8 head_dim), V scales
 * (head_dim), each in the order in which the lanes of a warp hold a
 * 16 x 16 tensor-core operand, so that attention reads a record straight into
 * its fragments.  With p = d / 64, w = (d / 16) mod 4 of element d:
 *   K, position m = 8 r + g:
 *     code  at  512 p + 16 (4 g + (d mod 16) / 4) + 8 r + 2 w + (d mod 4) / 2
 *     scale at  64 p + 8 g + 2 w + r
 *   V, position m = 8 ih + 2 t + il, i = 2 ih + il:
 *     code  at  512 p + 16 (4 ((d mod 16) / 2) + t) + 4 i + w
 *     scale at  64 p + 16 t + 4 w + i
 * with the code of an even d in the low half of its byte.
 *
 * A block's id is its index in the pool; a sequence's blocks are a row of
 * block_table[B][max_blocks] (int32): position p of sequence b lies in block
 * block_table[b][p / block_size], and its slot is that id * block_size + p mod
 * block_size.  One table serves all layers when their pools have the same
 * number of blocks.  Entries past a sequence's last block are not read; a
 * block id outside the pool is never dereferenced (its positions count as
 * absent in decode and as zeros in gather and prefill; the append does not
 * write them).  Blocks may be shared by several sequences as long as nobody
 * appends to them.
 *
 * head_dim, GQA groups, layer types, shared layers and errors are as above.
 * Layers are bf16 (G4_ERR_UNSUPPORTED otherwise).
 */

/*
 * One layer's pool, caller-owned device memory, 16-byte aligned:
 *   data        n_blocks * n_kv_heads * block_size / 16 * 18 * head_dim bytes
 *   block_size  16, 32, 64 or 128 positions
 *   k_exp       k is stored divided by 2^k_exp, -32 .. 32.  The e4m3 scales
 *               reach from 2^-9 to 448: 0 suits k_norm_w around 1; with k
 *               rows of another size take log2 of that size.
 * n_blocks * block_size must not exceed 2^31 - 1, and max_blocks * block_size of
 * a block table 2^30.  Layers that read another
 * layer's pool may leave their entry zeroed.
 */
typedef struct {
  void* data;
  int32_t layer_type;
  int32_t head_dim;
  int32_t n_kv_heads;
  int32_t n_blocks;
  int32_t block_size;
  int32_t k_exp;
} g4_kv4_pool;

/*
 * Gives the B sequences of a batch blocks of a pool as their lengths change,
 * and says where their new tokens go; one launch, no host round trip.
 *   old_lens, new_lens  [B] positions held now and wanted.  Growing takes
 *                   blocks, shrinking gives them back (new_lens 0: the
 *                   sequence has ended; old_lens 0: it is admitted).  Both are
 *                   clamped into [0, max_blocks * block_size], and a sequence
 *                   grows by T positions per call at most.
 *   free_blocks     [n_blocks] the pool's free block ids, free_count[0] of
 *                   them in front: a stack whose top is its last entry.
 *   block_table     [B][max_blocks]
 *   lens_out        [B] the lengths granted; may be old_lens itself
 *   free_count_out  [1]; may be free_count itself
 *   positions, slots  [B][T]: token t of sequence b is position old_lens[b]
 *                   + t and its slot, or -1 and -1 past its granted length
 *                   (g4_kv4_append_normrope's arguments).
 * Blocks given back are pushed first, in the order of sequences and entries
 * (an entry that holds no block of the pool, because the caller has taken it
 * away, gives none back); then blocks are popped in the same order.  Sequences are served first come,
 * first served: one that needs blocks is granted its new length if the
 * blocks of all sequences up to it fit, else it keeps old_lens and gets no
 * slots.  Writes the table entries of the blocks taken, at most as many
 * free_blocks entries behind the first free_count[0] as table entries are given
 * back, and the outputs; table entries of blocks given back keep their stale ids.  With lens_out and free_count_out apart from
 * the inputs, a repeated call (a replayed graph) repeats its results.  B is at
 * most 8192 and B * max_blocks, B * T at most 2^31 - 1.
 */
g4_status g4_kv4_assign_blocks(int32_t B, int32_t T, int32_t block_size, int32_t n_blocks, int32_t max_blocks,
                               const int32_t* old_lens, const int32_t* new_lens, int32_t* free_blocks,
                               const int32_t* free_count, int32_t* block_table, int32_t* lens_out,
                               int32_t* free_count_out, int32_t* positions, int32_t* slots, void* stream);

/*
 * g4_kv_append_normrope into a pool: q is normed and roped to q_out, k normed
 * and roped and v normed, and both stored in 4 bits at the tokens' slots.
 *   positions  [B][T] RoPE positions (any value)
 *   slots      [B][T] where k and v go; a slot outside the pool is not written
 * Other arguments as g4_kv_append_normrope; the layer's pool is pools[layer].
 * Two tokens of one call with the same slot leave a mixture of both rows.
 */
g4_status g4_kv4_append_normrope(const g4_layer_params* params, const g4_kv4_pool* pools, int32_t n_layers,
                                 int32_t layer, const void* q_in, const void* k_in, const void* v_in,
                                 const float* q_norm_w, const float* k_norm_w, const int32_t* positions,
                                 const int32_t* slots, int32_t B, int32_t T, void* q_out, void* stream);

/*
 * Reads positions [start[b], start[b] + rows) of every sequence back into
 * k_out, v_out [B][n_kv_heads][rows][head_dim] bf16, exactly the values the
 * pool stands for; zeros at positions from seq_lens[b] on (and below 0).  For
 * handing a context to the bf16 calls above, to another pool, or to the host.
 */
g4_status g4_kv4_gather(const g4_layer_params* params, const g4_kv4_pool* pools, int32_t n_layers, int32_t layer,
                        const int32_t* block_table, int32_t max_blocks, const int32_t* start,
                        const int32_t* seq_lens, int32_t B, int32_t rows, void* k_out, void* v_out, void* stream);

/* Workspace bytes g4_kv4_attn_decode needs (0: none). */
size_t g4_kv4_decode_workspace_size(const g4_layer_params* params, int32_t B, int32_t max_seq_len);

/*
 * g4_attn_decode over a pool: one query token per sequence.
 *   seq_lens     [B] keys per sequence including the new token (append it
 *                first), clamped into [0, max_seq_len].  A sequence of no
 *                keys gets an output of zeros.
 *   max_seq_len  1 .. max_blocks * block_size; B * n_kv_heads * max_seq_len (or
 *                the window) must stay below some 10^13 (G4_ERR_UNSUPPORTED)
 * q and out as g4_attn_decode.  The workspace is zero-filled once before its
 * first use; every call leaves it ready for the next, whatever that call's
 * layer, batch and lengths (size it for the largest).  Calls that overlap on
 * the GPU need a workspace each.  q.k and P.V run on
 * tensor cores from fp16 operands with float32 sums: keys and values are
 * exact in fp16, q is scaled by a power of two per head, and a probability and
 * its product with its value's scale are each rounded to fp16: relative to the
 * row's largest probability to 11 bits from 2^-18 on, below that to a multiple
 * of 2^-28.
 */
g4_status g4_kv4_attn_decode(const g4_layer_params* params, const g4_kv4_pool* pools, int32_t n_layers,
                             int32_t layer, const void* q, const int32_t* block_table, int32_t max_blocks,
                             const int32_t* seq_lens, int32_t B, int32_t max_seq_len, void* out, void* workspace,
                             size_t workspace_bytes, void* stream);

/* Workspace bytes g4_kv4_attn_prefill needs. */
size_t g4_kv4_prefill_workspace_size(const g4_layer_params* params, int32_t B, int32_t T, int32_t max_seq_len);

/*
 * g4_attn_prefill over a pool: T new tokens per sequence, token t of
 * sequence b at position q_start_pos[b] + t, appended before.
 *   seq_lens     [B] keys held, usually q_start_pos[b] + T.  Fewer (a padded
 *                batch) makes the tokens from seq_lens[b] - q_start_pos[b] on
 *                padding: their rows are computed as if the positions past
 *                seq_lens[b] held zero keys and values.
 *   max_seq_len  bound on seq_lens[b], T .. max_blocks * block_size.
 *                q_start_pos is clamped into [0, max_seq_len]; the padding of
 *                a sequence that ends near max_seq_len may lie past it
 *   workspace    16-byte aligned, no contents needed; not shared by calls
 *                that overlap
 * The keys that the T tokens see are laid out in the workspace as bf16 (a
 * sliding layer's T + window - 1, a full layer's max_seq_len + T per sequence: for
 * as many positions 3.6 times the pool's bytes, so max_seq_len is better the
 * longest length at hand than the longest there may be) and attention runs on the
 * tensor cores as in g4_attn_prefill, whose limits on launches in flight hold.  As
 * there, a masked key has the weight zero, and zero times NaN is NaN: a NaN or an
 * infinity held at a position may reach every query of the tiles (128 queries, 128
 * keys) that contain it.
 */
g4_status g4_kv4_attn_prefill(const g4_layer_params* params, const g4_kv4_pool* pools, int32_t n_layers,
                              int32_t layer, const void* q, const int32_t* block_table, int32_t max_blocks,
                              const int32_t* q_start_pos, const int32_t* seq_lens, int32_t B, int32_t T,
                              int32_t max_seq_len, void* out, void* workspace, size_t workspace_bytes,
                              void* stream);

/* ------------------------------------------------------------------------
 * Modified scores, intervals of keys, several position axes
 *
 * What prompts with images, rows packed of documents, padded batches and models
 * with capped or distance-biased scores need of the calls above.  (The pages have
 * no counterpart: these are calls of this library.)  Arrays of positions, lengths, ids,
 * intervals and slopes must be 4-byte aligned (G4_ERR_INVALID_ARG).
 */

/*
 * What is done to the scores of a layer.  With s = attn_scale q_i . k_j, in this
 * order:
 *   softcap    > 0: s becomes softcap tanh(s / softcap).  0: no cap.  Otherwise 2^-10
 *              .. 2^10 (G4_ERR_UNSUPPORTED outside).
 *              The bf16 prefill's scores are then off by up to 2^-20 of the cap: its weights
 *              by 5e-5 at a cap of 50, by 1e-3 (their bf16 rounding: 2e-3) at 2^10.
 *   slopes     [n_heads] float32 device, or NULL: s -= slopes[h] |i - j| (a bias that
 *              falls with distance in either direction).  Magnitudes up to 2^64; a key
 *              whose score is minus infinity weighs nothing.
 *   key_begin, key_end  int32 device, or NULL: query t of sequence b sees the
 *              positions key_begin[b][t] <= j < key_end[b][t] that the cache holds,
 *              whatever the layer's type and window say; g4_attn_visible_ranges makes
 *              both.  With key_begin NULL the interval begins where the layer's window
 *              does (at 0 on a full layer), with key_end NULL it ends with the query's own position.  A
 *              query whose interval is empty gets an output of zeros.
 * The arrays belong to the caller and are read by the kernels.
 */
typedef struct {
  float softcap;
  const float* slopes;
  const int32_t* key_begin;
  const int32_t* key_end;
} g4_score_mods;

/*
 * The interval of keys that each token sees, for g4_score_mods, from what a row
 * of positions is made of.  Token t of sequence b is position p = q_start_pos[b] + t.
 *   window       the sliding window of the layers that the intervals are for (>= 1), or
 *                0 for full layers
 *   q_start_pos  [B]
 *   seq_lens     [B] positions held, the new tokens among them
 *   doc_ids      [B][max_len] or NULL (one document): a document is a run of equal
 *                ids of neighbouring positions.  A token sees nothing before its
 *                document.  Below 0: padding, which sees nothing.
 *   span_ids     [B][max_len] or NULL (none): a run of equal ids >= 0 within a document is a span
 *                (an image, a prefix), whose tokens see all of it, in both directions and
 *                past the window.  Below 0: an ordinary token.
 *   max_len      row length of both, at most 2^24
 *   key_begin, key_end  [B][T].  With D the document's first position and S .. E the
 *                span's first and one past its last (at most seq_lens[b]):
 *                  key_begin = max(D, p - window + 1), key_end = p + 1,
 *                  in a span the smaller of that and S, and E.
 *                Both 0 (nothing) for tokens with p < 0, p >= seq_lens[b] or
 *                p >= max_len, and for padding.
 * Ids at positions from seq_lens[b] on are not read.  One call serves all layers of
 * the same window.
 */
g4_status g4_attn_visible_ranges(int32_t window, const int32_t* q_start_pos, const int32_t* seq_lens,
                                 const int32_t* doc_ids, const int32_t* span_ids, int32_t max_len, int32_t B, int32_t T,
                                 int32_t* key_begin, int32_t* key_end, void* stream);

/*
 * Positions of several axes (time, height and width of images and video).  Pair j is
 * dimensions j and j + head_dim / 2 of the whole head, as in g4_kv_append_normrope.  (Models
 * that give each axis a part of the head with halves of its own need their q and k
 * projections' rows, and norm weights, in that order: scores do not depend on it.)
 *   n_axes    1 .. 4
 *   axis      HOST [head_dim / 2]: the axis whose position turns pair j (pairs that
 *             rotary_fraction leaves unrotated are not looked at)
 *   inv_freq  HOST [head_dim / 2] or NULL: the frequency of pair j, 0 .. 1, instead of
 *             theta^(-2j / head_dim)
 * Both are read during the call.
 */
typedef struct {
  int32_t n_axes;
  const uint8_t* axis;
  const float* inv_freq;
} g4_rope_axes;

/*
 * g4_kv_append_normrope with positions of several axes, apart from the cache's:
 *   positions  [n_axes][B][T] RoPE positions (any value)
 *   rows       [B][T] the position that a token takes in the cache (NULL on a
 *              shared layer): as `positions` there, negative ones and, on a linear
 *              cache, those >= max_len are not written
 * Other arguments, and what is stored, as there: where all axes of a token agree
 * with its row, the same bits.
 */
g4_status g4_kv_append_normrope_axes(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                                     int32_t layer, const g4_rope_axes* axes, const void* q_in, const void* k_in,
                                     const void* v_in, const float* q_norm_w, const float* k_norm_w,
                                     const int32_t* positions, const int32_t* rows, int32_t B, int32_t T, void* q_out,
                                     void* stream);

/*
 * g4_attn_prefill with modified scores (mods NULL: none).  Arguments, caches, limits on
 * launches in flight and errors as there, with these differences:
 *   - q_start_pos is clamped into [0, 2^31 - 1 - T].
 *   - A position reaches the queries that see it and no others, whatever it holds: a
 *     padded batch's unwritten rows need no values, and a NaN or an infinity in one
 *     document stays there.  (bf16 rows of up to 32768 keys: those that share a tile with
 *     one that they do not see are formed again on CUDA cores, which takes long.
 *     Longer rows become NaN.)
 *   - On a ring, positions that it no longer holds count as absent; with key_begin
 *     NULL the window has to fit as there.
 */
g4_status g4_attn_prefill_mods(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                               int32_t layer, const g4_score_mods* mods, const void* q, const int32_t* q_start_pos,
                               int32_t B, int32_t T, void* out, void* stream);

/* Workspace bytes g4_attn_decode_mods needs (0: none). */
size_t g4_attn_decode_mods_workspace_size(const g4_layer_params* params, int32_t B, int32_t max_seq_len);

/*
 * g4_attn_decode with modified scores (mods NULL: none): the single-token form.
 * Arguments as there, with these differences:
 *   - seq_lens is clamped into [0, max_seq_len].
 *   - The workspace, zero-filled once before its first use, is left ready for the next
 *     call of this function, whatever that call's layer, batch and lengths (size it
 *     for the largest), also by one that g4_take_device_error reports as given up.
 *   - mods->key_begin is [B]: sequence b sees the keys [max(key_begin[b], its window's
 *     first), seq_lens[b]).  The new token is the last key: key_end must be NULL
 *     (G4_ERR_INVALID_ARG).  This is the interval that g4_attn_visible_ranges gives the
 *     token for T = 1, but in two cases:
 *       padding has the interval (0, 0), whose begin alone says "from 0": give such a
 *       sequence seq_lens[b] = 0 (or a key_begin[b] >= seq_lens[b]);
 *       a token in a span that begins before its layer's window sees the span's keys
 *       within the window only.
 *     g4_attn_prefill_mods with T = 1 takes the whole interval in both.
 *   - A sequence that sees no key gets an output of zeros.
 */
g4_status g4_attn_decode_mods(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                              int32_t layer, const g4_score_mods* mods, const void* q, const int32_t* seq_lens,
                              int32_t B, int32_t max_seq_len, void* out, void* workspace, size_t workspace_bytes,
                              void* stream);

/* Thread-local message of the last non-OK status ("" if none). */
const char* g4_last_error(void);

/*
 * Reads and clears the device-side error word (synchronises the device).
 * Nonzero means a kernel gave up a bounded wait (code 1), or found its
 * shared memory not 1024-byte aligned (code 2, the tensor-core prefill needs
 * that for its swizzled tiles), and returned early; its outputs are then
 * unspecified.  Returns -1 if the read itself failed.
 */
int32_t g4_take_device_error(void);

#ifdef __cplusplus
}
#endif

#endif /* G4ATTN_H */
