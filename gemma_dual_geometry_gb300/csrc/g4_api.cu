// C-ABI front end of libg4attn: argument validation, shared-KV source
// resolution, the float32 RoPE frequency table, and kernel dispatch.
// Declarations and the contract of every entry point: include/g4attn.h.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>
#include <string>

#include "../../include/g4attn.h"
#include "g4_kv4_internal.h"

namespace {

thread_local std::string g_last_error;

g4_status fail(g4_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
g4_status fail(g4_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

g4_status ok() {
  g_last_error.clear();
  return G4_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool supported_hd(int hd) { return hd == 64 || hd == 128 || hd == 256 || hd == 512; }

// Device error word: a kernel that gives up a bounded wait records a code here.
__device__ int g_device_error = 0;

// Its device address, looked up once per device (with that device current)
// under a lock, so host threads driving different GPUs each get their own.
int* device_error_ptr() {
  static std::mutex mu;
  static int* addr[128] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (addr[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
    addr[dev] = static_cast<int*>(p);
  }
  return addr[dev];
}

g4_status check_params(const g4_layer_params* p) {
  if (p == nullptr) return fail(G4_ERR_INVALID_ARG, "params is NULL");
  if (p->layer_type != G4_SLIDING && p->layer_type != G4_FULL)
    return fail(G4_ERR_INVALID_ARG, "layer_type %d is neither G4_SLIDING nor G4_FULL", p->layer_type);
  if (p->dtype != G4_F32 && p->dtype != G4_BF16) return fail(G4_ERR_INVALID_ARG, "dtype %d unknown", p->dtype);
  if (!supported_hd(p->head_dim))
    return fail(G4_ERR_UNSUPPORTED, "head_dim %d not supported (64, 128, 256, 512)", p->head_dim);
  if (p->n_heads < 1 || p->n_kv_heads < 1 || p->n_heads % p->n_kv_heads != 0)
    return fail(G4_ERR_INVALID_ARG, "n_heads %d must be a positive multiple of n_kv_heads %d", p->n_heads,
                p->n_kv_heads);
  const int g = p->n_heads / p->n_kv_heads;
  if (g != 1 && g != 2 && g != 4 && g != 8)
    return fail(G4_ERR_UNSUPPORTED, "GQA group %d not supported (1, 2, 4, 8)", g);
  if (g * p->head_dim > 2048)
    return fail(G4_ERR_UNSUPPORTED, "GQA group %d x head_dim %d exceeds 2048", g, p->head_dim);
  if (p->layer_type == G4_SLIDING && p->window < 1)
    return fail(G4_ERR_INVALID_ARG, "sliding layer needs window >= 1 (got %d)", p->window);
  if (!(p->theta > 0.0f) || !isfinite(p->theta)) return fail(G4_ERR_INVALID_ARG, "theta must be finite and > 0");
  if (!(p->rotary_fraction >= 0.0f && p->rotary_fraction <= 1.0f))
    return fail(G4_ERR_INVALID_ARG, "rotary_fraction must lie in [0, 1]");
  if (!(p->eps >= 0.0f) || !isfinite(p->eps)) return fail(G4_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!(p->attn_scale > 0.0f) || !isfinite(p->attn_scale))
    return fail(G4_ERR_INVALID_ARG, "attn_scale must be finite and > 0");
  return G4_OK;
}

// Resolves the cache a layer reads and checks that it matches the layer.
g4_status resolve_src(const g4_layer_params* p, const g4_kv_cache* caches, int n_layers, int layer,
                      const g4_kv_cache** out) {
  if (caches == nullptr) return fail(G4_ERR_INVALID_ARG, "caches is NULL");
  if (layer < 0 || layer >= n_layers) return fail(G4_ERR_INVALID_ARG, "layer %d outside [0, %d)", layer, n_layers);
  const int src = p->kv_share_src < 0 ? layer : p->kv_share_src;
  if (src >= n_layers) return fail(G4_ERR_INVALID_ARG, "kv_share_src %d outside [0, %d)", src, n_layers);
  const g4_kv_cache* c = &caches[src];
  if (c->k == nullptr || c->v == nullptr)
    return fail(G4_ERR_INVALID_ARG, "cache of layer %d (read by layer %d) has NULL k or v", src, layer);
  if (c->layer_type != p->layer_type || c->head_dim != p->head_dim || c->n_kv_heads != p->n_kv_heads ||
      c->dtype != p->dtype)
    return fail(G4_ERR_SHARE_MISMATCH,
                "layer %d (type %d, head_dim %d, n_kv %d, dtype %d) cannot read the cache of layer %d "
                "(type %d, head_dim %d, n_kv %d, dtype %d)",
                layer, p->layer_type, p->head_dim, p->n_kv_heads, p->dtype, src, c->layer_type, c->head_dim,
                c->n_kv_heads, c->dtype);
  if (c->max_len < 1 || c->batch < 1) return fail(G4_ERR_INVALID_ARG, "cache of layer %d has no rows", src);
  if (c->ring != 0 && c->ring != 1) return fail(G4_ERR_INVALID_ARG, "cache of layer %d: ring %d is neither 0 nor 1", src, c->ring);
  if (c->ring) {
    // A ring keeps the last max_len positions: only a sliding layer's window
    // fits in one, and the window itself must fit.
    if (c->layer_type != G4_SLIDING)
      return fail(G4_ERR_INVALID_ARG, "cache of layer %d is a ring but not a sliding layer's", src);
    if (c->max_len < p->window)
      return fail(G4_ERR_CAPACITY, "ring cache of layer %d has %d rows, fewer than the window %d", src, c->max_len,
                  p->window);
  }
  if (!aligned16(c->k) || !aligned16(c->v))
    return fail(G4_ERR_INVALID_ARG, "cache of layer %d is not 16-byte aligned", src);
  *out = c;
  return G4_OK;
}

// inv_freq[j] = theta^(-2j / hd) in float64, stored as float32, for the rotated
// pairs j < n_rot, zero past them.  The powers of a layer's constants take
// longer on the host than its launch, so a thread keeps the tables of the last
// few constants it has met (a stack alternates between two).
void rope_table(const g4_layer_params* p, int* n_rot_out, float* inv_freq) {
  struct Table {
    float theta;
    int hd, n_rot;
    float f[g4::kMaxHalf];
  };
  static thread_local Table kept[4] = {};
  static thread_local int oldest = 0;
  const int hd = p->head_dim, half = hd / 2;
  int n_rot = static_cast<int>(floor(static_cast<double>(hd) * static_cast<double>(p->rotary_fraction) / 2.0));
  if (n_rot > half) n_rot = half;
  *n_rot_out = n_rot;
  const Table* t = nullptr;
  for (const Table& k : kept)
    if (k.hd == hd && k.n_rot == n_rot && k.theta == p->theta) t = &k;
  if (t == nullptr) {
    Table* k = &kept[oldest];
    oldest = (oldest + 1) % 4;
    k->theta = p->theta;
    k->hd = hd;
    k->n_rot = n_rot;
    for (int j = 0; j < half; ++j)
      k->f[j] = j < n_rot ? static_cast<float>(pow(static_cast<double>(p->theta), -2.0 * j / hd)) : 0.0f;
    t = k;
  }
  memcpy(inv_freq, t->f, static_cast<size_t>(half) * sizeof(float));
}

g4_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ok();
  return fail(G4_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Scratch for g4_attn_decode_noalloc: a fixed array in device global memory,
// created when the library's device code is loaded on a GPU and held until the
// process exits.  Host code must not hand `g_noalloc_scratch` itself to a
// kernel (on the host it only names the symbol); noalloc_scratch() looks up
// its device address once per device.
constexpr size_t kNoAllocScratchBytes = G4_NOALLOC_SCRATCH_BYTES;
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

void* noalloc_scratch(cudaError_t* e) {
  static std::mutex mu;
  static void* addr[128] = {};
  int dev = 0;
  *e = cudaGetDevice(&dev);
  if (*e != cudaSuccess) return nullptr;
  if (dev < 0 || dev >= 128) {
    *e = cudaErrorInvalidDevice;
    return nullptr;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (addr[dev] == nullptr) {
    void* p = nullptr;
    *e = cudaGetSymbolAddress(&p, g_noalloc_scratch);  // with this device current
    if (*e != cudaSuccess) return nullptr;
    addr[dev] = p;
  }
  return addr[dev];
}

}  // namespace

extern "C" {

int32_t g4_kv_share_src(int32_t n_layers, int32_t n_shared, const int32_t* is_sliding, int32_t layer) {
  if (n_layers < 1 || n_shared < 0 || n_shared >= n_layers || is_sliding == nullptr || layer < 0 ||
      layer >= n_layers)
    return -2;
  const int first_shared = n_layers - n_shared;
  if (layer < first_shared) return -1;
  const int src = first_shared - (is_sliding[layer] ? 2 : 1);
  return src < 0 ? -2 : src;
}

g4_status g4_kv_append_normrope(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                                int32_t layer, const void* q_in, const void* k_in, const void* v_in,
                                const float* q_norm_w, const float* k_norm_w, const int32_t* positions, int32_t B,
                                int32_t T, void* q_out, void* stream) {
  g4_status st = check_params(params);
  if (st != G4_OK) return st;
  if (B < 0 || T < 0) return fail(G4_ERR_INVALID_ARG, "B %d and T %d must be >= 0", B, T);
  if (q_in == nullptr || q_out == nullptr || q_norm_w == nullptr || positions == nullptr)
    return fail(G4_ERR_INVALID_ARG, "q_in, q_out, q_norm_w and positions must be non-NULL");
  if (!aligned16(q_in) || !aligned16(q_out) || !aligned16(q_norm_w))
    return fail(G4_ERR_INVALID_ARG, "q_in, q_out and q_norm_w must be 16-byte aligned");
  const bool shared = params->kv_share_src >= 0;
  g4::AppendArgs a;
  memset(&a, 0, sizeof(a));
  if (shared) {
    if (k_in != nullptr || v_in != nullptr || k_norm_w != nullptr)
      return fail(G4_ERR_INVALID_ARG, "layer %d shares the cache of layer %d: k_in, v_in and k_norm_w must be NULL",
                  layer, params->kv_share_src);
    if (layer < 0 || layer >= n_layers) return fail(G4_ERR_INVALID_ARG, "layer %d outside [0, %d)", layer, n_layers);
  } else {
    if (k_in == nullptr || v_in == nullptr || k_norm_w == nullptr)
      return fail(G4_ERR_INVALID_ARG, "layer %d owns its cache: k_in, v_in and k_norm_w must be non-NULL", layer);
    if (!aligned16(k_in) || !aligned16(v_in) || !aligned16(k_norm_w))
      return fail(G4_ERR_INVALID_ARG, "k_in, v_in and k_norm_w must be 16-byte aligned");
    const g4_kv_cache* c = nullptr;
    st = resolve_src(params, caches, n_layers, layer, &c);
    if (st != G4_OK) return st;
    if (c->batch < B) return fail(G4_ERR_CAPACITY, "cache batch %d < B %d", c->batch, B);
    a.cache_k = c->k;
    a.cache_v = c->v;
    a.max_len = c->max_len;
    a.ring = c->ring;
    a.k_in = k_in;
    a.v_in = v_in;
    a.k_w = k_norm_w;
  }
  if (B == 0 || T == 0) return ok();
  a.q_in = q_in;
  a.q_w = q_norm_w;
  a.positions = positions;
  a.q_out = q_out;
  a.B = B;
  a.T = T;
  a.H = params->n_heads;
  a.Hkv = params->n_kv_heads;
  a.hd = params->head_dim;
  a.eps = params->eps;
  const int nrows = a.H + (shared ? 0 : 2 * a.Hkv);
  // Tokens at the same t of up to 8 sequences share a CTA (and, when their
  // positions agree, one cos/sin table); small launches split the rows.
  a.tok_per_cta = T >= 16 ? (B < 8 ? B : 8) : 1;
  const long long ctas = static_cast<long long>(T) * ((B + a.tok_per_cta - 1) / a.tok_per_cta);
  a.rows_per_cta = ctas >= 1024 ? nrows : 4;
  rope_table(params, &a.n_rot, a.inv_freq);
  return cuda_status(g4::launch_append(a, params->dtype, static_cast<cudaStream_t>(stream)), "append launch");
}

g4_status g4_attn_prefill(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                          int32_t layer, const void* q, const int32_t* q_start_pos, int32_t B, int32_t T,
                          void* out, void* stream) {
  g4_status st = check_params(params);
  if (st != G4_OK) return st;
  if (B < 0 || T < 0) return fail(G4_ERR_INVALID_ARG, "B %d and T %d must be >= 0", B, T);
  if (q == nullptr || out == nullptr || q_start_pos == nullptr)
    return fail(G4_ERR_INVALID_ARG, "q, out and q_start_pos must be non-NULL");
  if (!aligned16(q) || !aligned16(out)) return fail(G4_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  const g4_kv_cache* c = nullptr;
  st = resolve_src(params, caches, n_layers, layer, &c);
  if (st != G4_OK) return st;
  if (c->batch < B) return fail(G4_ERR_CAPACITY, "cache batch %d < B %d", c->batch, B);
  if (c->ring) {
    // Every key of the chunk's windows must still be in the ring after the
    // chunk's own T rows went in: T + window - 1 positions.
    if (static_cast<long long>(T) + params->window - 1 > c->max_len)
      return fail(G4_ERR_CAPACITY, "ring cache of %d rows cannot hold the %d + %d - 1 keys a chunk of T = %d needs",
                  c->max_len, T, params->window, T);
    if (params->dtype == G4_BF16 && c->max_len % 128 != 0)
      return fail(G4_ERR_UNSUPPORTED, "bf16 prefill on a ring cache needs max_len a multiple of 128 (got %d)",
                  c->max_len);
  } else if (T > c->max_len) {
    return fail(G4_ERR_CAPACITY, "T %d exceeds the cache length %d", T, c->max_len);
  }
  if (B == 0 || T == 0) return ok();
  int* err = device_error_ptr();
  if (err == nullptr) return fail(G4_ERR_CUDA, "cannot resolve the device error word");
  const float scale_log2 = params->attn_scale * 1.4426950408889634f;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (params->dtype == G4_BF16) {
    g4::PrefillTcArgs a;
    memset(&a, 0, sizeof(a));
    a.q = q;
    a.ck = c->k;
    a.cv = c->v;
    a.out = out;
    a.q_start = q_start_pos;
    a.err = err;
    a.B = B;
    a.T = T;
    a.H = params->n_heads;
    a.Hkv = params->n_kv_heads;
    a.hd = params->head_dim;
    a.max_len = c->max_len;
    a.ring = c->ring;
    a.sliding = params->layer_type == G4_SLIDING;
    a.window = params->window;
    a.scale_log2 = scale_log2;
    return cuda_status(g4::launch_prefill_tc(a, s), "tcgen05 prefill launch");
  }
  g4::AttnSimtArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.ck = c->k;
  a.cv = c->v;
  a.out = out;
  a.base = q_start_pos;
  a.err = err;
  a.mode = 1;
  a.B = B;
  a.T = T;
  a.H = params->n_heads;
  a.Hkv = params->n_kv_heads;
  a.hd = params->head_dim;
  a.max_len = c->max_len;
  a.ring = c->ring;
  a.sliding = params->layer_type == G4_SLIDING;
  a.window = params->window;
  a.len_cap = c->max_len;
  a.chunk = a.sliding ? params->window : c->max_len;
  a.nsplit = 1;
  a.scale_log2 = scale_log2;
  return cuda_status(g4::launch_attn_simt(a, params->dtype, s), "float32 prefill launch");
}

g4_status g4_attn_encoder(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                          int32_t layer, const void* q, int32_t B, int32_t T, void* out, void* stream) {
  g4_status st = check_params(params);
  if (st != G4_OK) return st;
  if (B < 0 || T < 0) return fail(G4_ERR_INVALID_ARG, "B %d and T %d must be >= 0", B, T);
  if (q == nullptr || out == nullptr) return fail(G4_ERR_INVALID_ARG, "q and out must be non-NULL");
  if (!aligned16(q) || !aligned16(out)) return fail(G4_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  const g4_kv_cache* c = nullptr;
  st = resolve_src(params, caches, n_layers, layer, &c);
  if (st != G4_OK) return st;
  if (c->ring)
    return fail(G4_ERR_INVALID_ARG, "the encoder reads the sequence's keys at rows 0 .. T-1: a ring cache cannot hold them");
  if (c->batch < B) return fail(G4_ERR_CAPACITY, "cache batch %d < B %d", c->batch, B);
  if (T > c->max_len) return fail(G4_ERR_CAPACITY, "T %d exceeds the cache length %d", T, c->max_len);
  if (B == 0 || T == 0) return ok();
  int* err = device_error_ptr();
  if (err == nullptr) return fail(G4_ERR_CUDA, "cannot resolve the device error word");
  const bool sliding = params->layer_type == G4_SLIDING;
  // A window of T or more keys reaches every key; capping it keeps i + window
  // in range.
  const int window = sliding ? (params->window < T ? params->window : T) : 0;
  const float scale_log2 = params->attn_scale * 1.4426950408889634f;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (params->dtype == G4_BF16) {
    g4::PrefillTcArgs a;
    memset(&a, 0, sizeof(a));
    a.q = q;
    a.ck = c->k;
    a.cv = c->v;
    a.out = out;
    a.q_start = nullptr;  // unused: token t sits at position t
    a.err = err;
    a.B = B;
    a.T = T;
    a.H = params->n_heads;
    a.Hkv = params->n_kv_heads;
    a.hd = params->head_dim;
    a.max_len = c->max_len;
    a.sliding = sliding;
    a.window = window;
    a.bidir = 1;
    a.scale_log2 = scale_log2;
    return cuda_status(g4::launch_prefill_tc(a, s), "tcgen05 encoder launch");
  }
  g4::AttnSimtArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.ck = c->k;
  a.cv = c->v;
  a.out = out;
  a.err = err;
  a.mode = 2;
  a.B = B;
  a.T = T;
  a.H = params->n_heads;
  a.Hkv = params->n_kv_heads;
  a.hd = params->head_dim;
  a.max_len = c->max_len;
  a.sliding = sliding;
  a.window = window;
  a.len_cap = c->max_len;
  // one split holds a query's whole key range (2 window + 1 keys at most, T at most)
  a.chunk = sliding && 2LL * window + 1 < T ? 2 * window + 1 : T;
  a.nsplit = 1;
  a.scale_log2 = scale_log2;
  return cuda_status(g4::launch_attn_simt(a, params->dtype, s), "float32 encoder launch");
}

size_t g4_attn_decode_workspace_size(const g4_layer_params* params, int32_t B, int32_t max_seq_len) {
  if (check_params(params) != G4_OK || B < 1 || max_seq_len < 1) return 0;
  return g4::decode_plan(params->dtype, params->layer_type == G4_SLIDING, params->window, params->head_dim, params->n_heads,
                         params->n_kv_heads, B, max_seq_len)
      .ws_bytes;
}

}  // extern "C"

namespace {

// Shared by g4_attn_decode and g4_decode_step: validation, split plan and launch.
// q is normed+roped (fused == false) or the raw projection (fused == true, with
// k_in / v_in / weights and the RoPE table of the layer).
// With clear_tickets the splits' arrival counters in the workspace are
// zeroed on the stream right before the launch, after every check passed
// (the built-in scratch of g4_attn_decode_noalloc; a caller's workspace is
// left zeroed by the previous call instead).
g4_status decode_common(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers, int32_t layer,
                        const void* q, const void* k_in, const void* v_in, const float* q_norm_w,
                        const float* k_norm_w, bool fused, const int32_t* seq_lens, int32_t B, int32_t max_seq_len,
                        void* out, void* workspace, size_t workspace_bytes, void* stream,
                        bool clear_tickets = false) {
  g4_status st = check_params(params);
  if (st != G4_OK) return st;
  if (B < 0) return fail(G4_ERR_INVALID_ARG, "B %d must be >= 0", B);
  if (q == nullptr || out == nullptr || seq_lens == nullptr)
    return fail(G4_ERR_INVALID_ARG, "q, out and seq_lens must be non-NULL");
  if (!aligned16(q) || !aligned16(out)) return fail(G4_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  const bool shared = params->kv_share_src >= 0;
  if (fused) {
    if (q_norm_w == nullptr || !aligned16(q_norm_w))
      return fail(G4_ERR_INVALID_ARG, "q_norm_w must be non-NULL and 16-byte aligned");
    if (shared && (k_in != nullptr || v_in != nullptr || k_norm_w != nullptr))
      return fail(G4_ERR_INVALID_ARG, "layer %d shares the cache of layer %d: k_in, v_in and k_norm_w must be NULL",
                  layer, params->kv_share_src);
    if (!shared && (k_in == nullptr || v_in == nullptr || k_norm_w == nullptr))
      return fail(G4_ERR_INVALID_ARG, "layer %d owns its cache: k_in, v_in and k_norm_w must be non-NULL", layer);
    if (!shared && (!aligned16(k_in) || !aligned16(v_in) || !aligned16(k_norm_w)))
      return fail(G4_ERR_INVALID_ARG, "k_in, v_in and k_norm_w must be 16-byte aligned");
  }
  const g4_kv_cache* c = nullptr;
  st = resolve_src(params, caches, n_layers, layer, &c);
  if (st != G4_OK) return st;
  if (c->batch < B) return fail(G4_ERR_CAPACITY, "cache batch %d < B %d", c->batch, B);
  if (max_seq_len < 1 || (!c->ring && max_seq_len > c->max_len))
    return fail(G4_ERR_CAPACITY, "max_seq_len %d outside [1, cache length %d]", max_seq_len, c->max_len);
  if (B == 0) return ok();
  const g4::DecodePlan plan = g4::decode_plan(params->dtype, params->layer_type == G4_SLIDING, params->window, params->head_dim,
                                              params->n_heads, params->n_kv_heads, B, max_seq_len);
  if (workspace_bytes < plan.ws_bytes)
    return fail(G4_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed", workspace_bytes, plan.ws_bytes);
  if (plan.ws_bytes > 0 && (workspace == nullptr || !aligned16(workspace)))
    return fail(G4_ERR_INVALID_ARG, "workspace must be non-NULL and 16-byte aligned");
  int* err = device_error_ptr();
  if (err == nullptr) return fail(G4_ERR_CUDA, "cannot resolve the device error word");
  g4::AttnSimtArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.ck = c->k;
  a.cv = c->v;
  a.out = out;
  a.base = seq_lens;
  a.err = err;
  a.mode = 0;
  a.B = B;
  a.T = 1;
  a.H = params->n_heads;
  a.Hkv = params->n_kv_heads;
  a.hd = params->head_dim;
  a.max_len = c->max_len;
  a.ring = c->ring;
  a.sliding = params->layer_type == G4_SLIDING;
  a.window = params->window;
  a.len_cap = max_seq_len;
  a.chunk = plan.chunk;
  a.nsplit = plan.nsplit;
  a.scale_log2 = params->attn_scale * 1.4426950408889634f;
  if (plan.nsplit > 1) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.ws_o = reinterpret_cast<float*>(ws);
    a.ws_m = reinterpret_cast<float*>(ws + plan.o_bytes);
    a.ws_l = reinterpret_cast<float*>(ws + plan.o_bytes + plan.m_bytes);
    a.tickets = reinterpret_cast<unsigned*>(ws + plan.o_bytes + 2 * plan.m_bytes);
    if (clear_tickets) {
      const cudaError_t e = cudaMemsetAsync(a.tickets, 0, plan.t_bytes, static_cast<cudaStream_t>(stream));
      if (e != cudaSuccess) return cuda_status(e, "clearing the decode scratch's arrival counters");
    }
  }
  if (fused) {
    a.fused = 1;
    a.q_w = q_norm_w;
    a.eps = params->eps;
    if (!shared) {
      a.k_raw = k_in;
      a.v_raw = v_in;
      a.k_w = k_norm_w;
      a.cache_k = caches[layer].k;
      a.cache_v = caches[layer].v;
    }
    rope_table(params, &a.n_rot, a.inv_freq);
  }
  if (plan.win)
    return cuda_status(g4::launch_decode_win(a, static_cast<cudaStream_t>(stream)), "windowed decode launch");
  return cuda_status(g4::launch_attn_simt(a, params->dtype, static_cast<cudaStream_t>(stream)), "decode launch");
}

}  // namespace

extern "C" {

g4_status g4_attn_decode(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers, int32_t layer,
                         const void* q, const int32_t* seq_lens, int32_t B, int32_t max_seq_len, void* out,
                         void* workspace, size_t workspace_bytes, void* stream) {
  return decode_common(params, caches, n_layers, layer, q, nullptr, nullptr, nullptr, nullptr, false, seq_lens, B,
                       max_seq_len, out, workspace, workspace_bytes, stream);
}

g4_status g4_decode_step(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers, int32_t layer,
                         const void* q_in, const void* k_in, const void* v_in, const float* q_norm_w,
                         const float* k_norm_w, const int32_t* seq_lens, int32_t B, int32_t max_seq_len, void* out,
                         void* workspace, size_t workspace_bytes, void* stream) {
  return decode_common(params, caches, n_layers, layer, q_in, k_in, v_in, q_norm_w, k_norm_w, true, seq_lens, B,
                       max_seq_len, out, workspace, workspace_bytes, stream);
}

g4_status g4_attn_decode_noalloc(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                                 int32_t layer, const void* q, const int32_t* seq_lens, int32_t B,
                                 int32_t max_seq_len, void* out, void* stream) {
  g4_status st = check_params(params);
  if (st != G4_OK) return st;
  if (B >= 1 && max_seq_len >= 1) {
    const g4::DecodePlan plan = g4::decode_plan(params->dtype, params->layer_type == G4_SLIDING, params->window,
                                                params->head_dim, params->n_heads, params->n_kv_heads, B,
                                                max_seq_len);
    if (plan.ws_bytes > kNoAllocScratchBytes)
      return fail(G4_ERR_WORKSPACE,
                  "this decode needs %zu bytes of scratch, more than the %zu bytes built into the library for "
                  "g4_attn_decode_noalloc; call g4_attn_decode with a caller-allocated workspace instead",
                  plan.ws_bytes, kNoAllocScratchBytes);
  }
  cudaError_t e = cudaSuccess;
  void* scratch = noalloc_scratch(&e);
  if (scratch == nullptr) return fail(G4_ERR_CUDA, "cannot resolve the built-in decode scratch: %s", cudaGetErrorString(e));
  // Same kernels and split plan as g4_attn_decode, with the split partials in
  // the built-in array.  The partials are written before they are read; the
  // splits' arrival counters must start at zero, so decode_common clears them
  // once every argument has been checked, just before the launch.
  return decode_common(params, caches, n_layers, layer, q, nullptr, nullptr, nullptr, nullptr, false, seq_lens, B,
                       max_seq_len, out, scratch, kNoAllocScratchBytes, stream, /*clear_tickets=*/true);
}

g4_status g4_qkv_project_append(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                                int32_t layer, const void* x, int32_t D, const void* w_qkv, const float* q_norm_w,
                                const float* k_norm_w, const int32_t* positions, int32_t B, int32_t T, void* q_out,
                                void* stream) {
  g4_status st = check_params(params);
  if (st != G4_OK) return st;
  if (params->dtype != G4_BF16)
    return fail(G4_ERR_UNSUPPORTED, "the fused projection runs on the bf16 tensor cores only");
  if (B < 0 || T < 0) return fail(G4_ERR_INVALID_ARG, "B %d and T %d must be >= 0", B, T);
  if (D < 64 || D % 64 != 0) return fail(G4_ERR_UNSUPPORTED, "D %d must be a positive multiple of 64", D);
  if (x == nullptr || w_qkv == nullptr || q_norm_w == nullptr || positions == nullptr || q_out == nullptr)
    return fail(G4_ERR_INVALID_ARG, "x, w_qkv, q_norm_w, positions and q_out must be non-NULL");
  if (!aligned16(x) || !aligned16(w_qkv) || !aligned16(q_out) || !aligned16(q_norm_w))
    return fail(G4_ERR_INVALID_ARG, "x, w_qkv, q_norm_w and q_out must be 16-byte aligned");
  const bool shared = params->kv_share_src >= 0;
  g4::GemmArgs a;
  memset(&a, 0, sizeof(a));
  if (shared) {
    if (k_norm_w != nullptr)
      return fail(G4_ERR_INVALID_ARG, "layer %d shares the cache of layer %d: k_norm_w must be NULL", layer,
                  params->kv_share_src);
    if (layer < 0 || layer >= n_layers) return fail(G4_ERR_INVALID_ARG, "layer %d outside [0, %d)", layer, n_layers);
  } else {
    if (k_norm_w == nullptr || !aligned16(k_norm_w))
      return fail(G4_ERR_INVALID_ARG, "layer %d owns its cache: k_norm_w must be non-NULL and 16-byte aligned", layer);
    const g4_kv_cache* c = nullptr;
    st = resolve_src(params, caches, n_layers, layer, &c);
    if (st != G4_OK) return st;
    if (c->batch < B) return fail(G4_ERR_CAPACITY, "cache batch %d < B %d", c->batch, B);
    a.cache_k = c->k;
    a.cache_v = c->v;
    a.max_len = c->max_len;
    a.ring = c->ring;
    a.k_w = k_norm_w;
  }
  const long long M = static_cast<long long>(B) * T;
  if (M == 0) return ok();
  if (M > 0x7fffffffLL - 128) return fail(G4_ERR_INVALID_ARG, "B * T too large");
  const int hd = params->head_dim;
  a.epi = 0;
  a.M = static_cast<int>(M);
  a.K = D;
  a.N = (params->n_heads + (shared ? 0 : 2 * params->n_kv_heads)) * hd;
  a.B = B;
  a.T = T;
  a.H = params->n_heads;
  a.Hkv = params->n_kv_heads;
  a.hd = hd;
  a.eps = params->eps;
  a.eps_in = params->eps;
  a.q_w = q_norm_w;
  a.positions = positions;
  a.q_out = q_out;
  rope_table(params, &a.n_rot, a.inv_freq);
  int* err = device_error_ptr();
  if (err == nullptr) return fail(G4_ERR_CUDA, "cannot resolve the device error word");
  a.err = err;
  return cuda_status(g4::launch_gemm_tc(a, x, w_qkv, static_cast<cudaStream_t>(stream)), "projection launch");
}

g4_status g4_attn_out_residual(const void* ao, int32_t M, int32_t K, const void* w_o, int32_t D,
                               const float* post_norm_w, float eps, const void* h, void* out, void* stream) {
  if (M < 0) return fail(G4_ERR_INVALID_ARG, "M %d must be >= 0", M);
  if (K < 64 || K % 64 != 0) return fail(G4_ERR_UNSUPPORTED, "K %d must be a positive multiple of 64", K);
  if (D < 256 || D % 256 != 0 || D > 2048)
    return fail(G4_ERR_UNSUPPORTED, "D %d must be a multiple of 256 in [256, 2048]", D);
  if (!(eps >= 0.0f) || !isfinite(eps)) return fail(G4_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (ao == nullptr || w_o == nullptr || post_norm_w == nullptr || h == nullptr || out == nullptr)
    return fail(G4_ERR_INVALID_ARG, "ao, w_o, post_norm_w, h and out must be non-NULL");
  if (!aligned16(ao) || !aligned16(w_o) || !aligned16(h) || !aligned16(out))
    return fail(G4_ERR_INVALID_ARG, "ao, w_o, h and out must be 16-byte aligned");
  if (M == 0) return ok();
  if (M > 0x7fffffff - 128) return fail(G4_ERR_INVALID_ARG, "M too large");
  int* err = device_error_ptr();
  if (err == nullptr) return fail(G4_ERR_CUDA, "cannot resolve the device error word");
  g4::GemmArgs a;
  memset(&a, 0, sizeof(a));
  a.epi = 1;
  a.M = M;
  a.K = K;
  a.N = D;
  a.err = err;
  a.eps = eps;
  a.h = h;
  a.out = out;
  a.post_w = post_norm_w;
  return cuda_status(g4::launch_gemm_tc(a, ao, w_o, static_cast<cudaStream_t>(stream)), "o_proj launch");
}

}  // extern "C"

namespace {

// Positions of a table's row at most: sums of a length and a few blocks stay in 32 bits.
constexpr long long kKv4MaxLen = 1LL << 30;

bool kv4_block_size(int bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }
int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

// check_params, and what the 4-bit cache adds to it.
g4_status kv4_check_params(const g4_layer_params* p) {
  const g4_status st = check_params(p);
  if (st != G4_OK) return st;
  if (p->dtype != G4_BF16) return fail(G4_ERR_UNSUPPORTED, "the 4-bit cache serves bf16 layers only");
  return G4_OK;
}

// Resolves the pool a layer reads and checks that it matches the layer.
g4_status kv4_resolve_src(const g4_layer_params* p, const g4_kv4_pool* pools, int n_layers, int layer,
                          const g4_kv4_pool** out) {
  if (pools == nullptr) return fail(G4_ERR_INVALID_ARG, "pools is NULL");
  if (layer < 0 || layer >= n_layers) return fail(G4_ERR_INVALID_ARG, "layer %d outside [0, %d)", layer, n_layers);
  const int src = p->kv_share_src < 0 ? layer : p->kv_share_src;
  if (src >= n_layers) return fail(G4_ERR_INVALID_ARG, "kv_share_src %d outside [0, %d)", src, n_layers);
  const g4_kv4_pool* c = &pools[src];
  if (c->data == nullptr) return fail(G4_ERR_INVALID_ARG, "pool of layer %d (read by layer %d) has NULL data", src, layer);
  if (c->layer_type != p->layer_type || c->head_dim != p->head_dim || c->n_kv_heads != p->n_kv_heads)
    return fail(G4_ERR_SHARE_MISMATCH,
                "layer %d (type %d, head_dim %d, n_kv %d) cannot read the pool of layer %d (type %d, head_dim %d, n_kv %d)",
                layer, p->layer_type, p->head_dim, p->n_kv_heads, src, c->layer_type, c->head_dim, c->n_kv_heads);
  if (!kv4_block_size(c->block_size))
    return fail(G4_ERR_UNSUPPORTED, "pool of layer %d: block_size %d not supported (16, 32, 64, 128)", src, c->block_size);
  if (c->n_blocks < 1 || static_cast<long long>(c->n_blocks) * c->block_size > 0x7fffffffLL)
    return fail(G4_ERR_INVALID_ARG, "pool of layer %d: %d blocks of %d positions outside [1, 2^31 - 1] positions", src,
                c->n_blocks, c->block_size);
  if (c->k_exp < -32 || c->k_exp > 32)
    return fail(G4_ERR_INVALID_ARG, "pool of layer %d: k_exp %d outside [-32, 32]", src, c->k_exp);
  if (!aligned16(c->data)) return fail(G4_ERR_INVALID_ARG, "pool of layer %d is not 16-byte aligned", src);
  *out = c;
  return G4_OK;
}

// The table's width against a pool's block size (max_blocks * block_size is a length).
g4_status kv4_check_table(const void* table, int max_blocks, int block_size) {
  if (table == nullptr) return fail(G4_ERR_INVALID_ARG, "block_table must be non-NULL");
  if (max_blocks < 1 || static_cast<long long>(max_blocks) * block_size > kKv4MaxLen)
    return fail(G4_ERR_INVALID_ARG, "max_blocks %d outside [1, 2^30 / %d]", max_blocks, block_size);
  return G4_OK;
}

// The bf16 rows that a prefill's keys are laid out in: per sequence, and the bytes of K (as of V).
// (T tokens from max_seq_len on at most, the padding of a padded batch; T + max_seq_len < 2^31.)
int kv4_prefill_rows(const g4_layer_params* p, int T, int max_seq_len) {
  const int all = max_seq_len + T;
  if (p->layer_type != G4_SLIDING) return all;
  const long long rows = static_cast<long long>(T) + p->window - 1;
  return rows < all ? static_cast<int>(rows) : all;
}
size_t kv4_prefill_kv_bytes(const g4_layer_params* p, int B, int T, int max_seq_len) {
  return static_cast<size_t>(B) * p->n_kv_heads * kv4_prefill_rows(p, T, max_seq_len) * p->head_dim * 2;
}
size_t kv4_prefill_head_bytes(int B) { return (static_cast<size_t>(B) * 4 + 255) / 256 * 256; }

}  // namespace

extern "C" {

g4_status g4_kv4_assign_blocks(int32_t B, int32_t T, int32_t block_size, int32_t n_blocks, int32_t max_blocks,
                               const int32_t* old_lens, const int32_t* new_lens, int32_t* free_blocks,
                               const int32_t* free_count, int32_t* block_table, int32_t* lens_out,
                               int32_t* free_count_out, int32_t* positions, int32_t* slots, void* stream) {
  if (B < 0 || T < 0) return fail(G4_ERR_INVALID_ARG, "B %d and T %d must be >= 0", B, T);
  if (!kv4_block_size(block_size))
    return fail(G4_ERR_UNSUPPORTED, "block_size %d not supported (16, 32, 64, 128)", block_size);
  if (n_blocks < 1 || static_cast<long long>(n_blocks) * block_size > 0x7fffffffLL)
    return fail(G4_ERR_INVALID_ARG, "%d blocks of %d positions outside [1, 2^31 - 1] positions", n_blocks, block_size);
  if (max_blocks < 1 || static_cast<long long>(max_blocks) * block_size > kKv4MaxLen)
    return fail(G4_ERR_INVALID_ARG, "max_blocks %d outside [1, 2^30 / %d]", max_blocks, block_size);
  if (B > g4::kKv4MaxBatch)
    return fail(G4_ERR_UNSUPPORTED, "B %d exceeds %d sequences", B, g4::kKv4MaxBatch);
  if (static_cast<long long>(B) * max_blocks > 0x7fffffffLL || static_cast<long long>(B) * T > 0x7fffffffLL)
    return fail(G4_ERR_INVALID_ARG, "B * max_blocks and B * T must not exceed 2^31 - 1");
  if (old_lens == nullptr || new_lens == nullptr || free_blocks == nullptr || free_count == nullptr ||
      block_table == nullptr || lens_out == nullptr || free_count_out == nullptr)
    return fail(G4_ERR_INVALID_ARG, "lengths, free list, table and their outputs must be non-NULL");
  if (T > 0 && (positions == nullptr || slots == nullptr))
    return fail(G4_ERR_INVALID_ARG, "positions and slots must be non-NULL");
  // (B = 0 still passes the count on)
  g4::Kv4AssignArgs a;
  memset(&a, 0, sizeof(a));
  a.B = B;
  a.T = T;
  a.block_shift = log2_of(block_size);
  a.n_blocks = n_blocks;
  a.max_blocks = max_blocks;
  a.old_lens = old_lens;
  a.new_lens = new_lens;
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.table = block_table;
  a.lens_out = lens_out;
  a.count_out = free_count_out;
  a.positions = positions;
  a.slots = slots;
  return cuda_status(g4::launch_kv4_assign(a, static_cast<cudaStream_t>(stream)), "block assignment launch");
}

g4_status g4_kv4_append_normrope(const g4_layer_params* params, const g4_kv4_pool* pools, int32_t n_layers,
                                 int32_t layer, const void* q_in, const void* k_in, const void* v_in,
                                 const float* q_norm_w, const float* k_norm_w, const int32_t* positions,
                                 const int32_t* slots, int32_t B, int32_t T, void* q_out, void* stream) {
  g4_status st = kv4_check_params(params);
  if (st != G4_OK) return st;
  if (B < 0 || T < 0) return fail(G4_ERR_INVALID_ARG, "B %d and T %d must be >= 0", B, T);
  if (q_in == nullptr || q_out == nullptr || q_norm_w == nullptr || positions == nullptr)
    return fail(G4_ERR_INVALID_ARG, "q_in, q_out, q_norm_w and positions must be non-NULL");
  if (!aligned16(q_in) || !aligned16(q_out) || !aligned16(q_norm_w))
    return fail(G4_ERR_INVALID_ARG, "q_in, q_out and q_norm_w must be 16-byte aligned");
  const bool shared = params->kv_share_src >= 0;
  g4::Kv4AppendArgs a;
  memset(&a, 0, sizeof(a));
  if (shared) {
    if (k_in != nullptr || v_in != nullptr || k_norm_w != nullptr)
      return fail(G4_ERR_INVALID_ARG, "layer %d shares the pool of layer %d: k_in, v_in and k_norm_w must be NULL",
                  layer, params->kv_share_src);
    if (layer < 0 || layer >= n_layers) return fail(G4_ERR_INVALID_ARG, "layer %d outside [0, %d)", layer, n_layers);
  } else {
    if (k_in == nullptr || v_in == nullptr || k_norm_w == nullptr || slots == nullptr)
      return fail(G4_ERR_INVALID_ARG, "layer %d owns its pool: k_in, v_in, k_norm_w and slots must be non-NULL", layer);
    if (!aligned16(k_in) || !aligned16(v_in) || !aligned16(k_norm_w))
      return fail(G4_ERR_INVALID_ARG, "k_in, v_in and k_norm_w must be 16-byte aligned");
    const g4_kv4_pool* c = nullptr;
    st = kv4_resolve_src(params, pools, n_layers, layer, &c);
    if (st != G4_OK) return st;
    a.cache_k = c->data;
    a.n_slots = c->n_blocks * c->block_size;
    a.block_shift = log2_of(c->block_size);
    a.k_mul = static_cast<float>(ldexp(1.0, -c->k_exp));
    a.k_in = k_in;
    a.v_in = v_in;
    a.k_w = k_norm_w;
    a.slots = slots;
  }
  const long long tokens = static_cast<long long>(B) * T;
  if (tokens > 0x7fffffffLL) return fail(G4_ERR_INVALID_ARG, "B * T exceeds 2^31 - 1");
  if (tokens == 0) return ok();
  a.q_in = q_in;
  a.q_w = q_norm_w;
  a.positions = positions;
  a.q_out = q_out;
  a.B = B;
  a.T = T;
  a.H = params->n_heads;
  a.Hkv = params->n_kv_heads;
  a.hd = params->head_dim;
  a.eps = params->eps;
  // Tokens at the same t of a few sequences share a CTA (and, where their
  // positions agree, a cos/sin table); small launches split the rows.  4 tokens
  // measured 1-4 % faster than 8 (whose CTAs are fewer than three waves at
  // 8 x 2048 tokens) and 10 % faster than 1 (no rows to load ahead).
  const int nrows = a.H + (shared ? 0 : 2 * a.Hkv);
  a.tok_per_cta = T >= 16 ? (B < g4::kAppendMaxTokens ? B : g4::kAppendMaxTokens) : 1;
  const long long ctas = static_cast<long long>(T) * ((B + a.tok_per_cta - 1) / a.tok_per_cta);
  a.rows_per_cta = ctas >= 1024 ? nrows : 4;
  rope_table(params, &a.n_rot, a.inv_freq);
  return cuda_status(g4::launch_kv4_append(a, static_cast<cudaStream_t>(stream)), "4-bit append launch");
}

g4_status g4_kv4_gather(const g4_layer_params* params, const g4_kv4_pool* pools, int32_t n_layers, int32_t layer,
                        const int32_t* block_table, int32_t max_blocks, const int32_t* start,
                        const int32_t* seq_lens, int32_t B, int32_t rows, void* k_out, void* v_out, void* stream) {
  g4_status st = kv4_check_params(params);
  if (st != G4_OK) return st;
  if (B < 0 || rows < 0) return fail(G4_ERR_INVALID_ARG, "B %d and rows %d must be >= 0", B, rows);
  if (start == nullptr || seq_lens == nullptr || k_out == nullptr || v_out == nullptr)
    return fail(G4_ERR_INVALID_ARG, "start, seq_lens, k_out and v_out must be non-NULL");
  if (!aligned16(k_out) || !aligned16(v_out))
    return fail(G4_ERR_INVALID_ARG, "k_out and v_out must be 16-byte aligned");
  const g4_kv4_pool* c = nullptr;
  st = kv4_resolve_src(params, pools, n_layers, layer, &c);
  if (st != G4_OK) return st;
  st = kv4_check_table(block_table, max_blocks, c->block_size);
  if (st != G4_OK) return st;
  if (B == 0 || rows == 0) return ok();
  g4::Kv4GatherArgs a;
  memset(&a, 0, sizeof(a));
  a.data = static_cast<const uint8_t*>(c->data);
  a.table = block_table;
  a.start = start;
  a.lens = seq_lens;
  a.k = k_out;
  a.v = v_out;
  a.B = B;
  a.Hkv = params->n_kv_heads;
  a.hd = params->head_dim;
  a.rows = rows;
  a.max_blocks = max_blocks;
  a.n_blocks = c->n_blocks;
  a.block_shift = log2_of(c->block_size);
  a.k_mul = static_cast<float>(ldexp(1.0, c->k_exp));
  return cuda_status(g4::launch_kv4_gather(a, static_cast<cudaStream_t>(stream)), "4-bit gather launch");
}

size_t g4_kv4_decode_workspace_size(const g4_layer_params* params, int32_t B, int32_t max_seq_len) {
  if (kv4_check_params(params) != G4_OK || B < 1 || max_seq_len < 1) return 0;
  return g4::kv4_decode_plan(params->layer_type == G4_SLIDING ? params->window : 0, params->head_dim, params->n_heads,
                             params->n_kv_heads, B, max_seq_len)
      .ws_bytes;
}

g4_status g4_kv4_attn_decode(const g4_layer_params* params, const g4_kv4_pool* pools, int32_t n_layers,
                             int32_t layer, const void* q, const int32_t* block_table, int32_t max_blocks,
                             const int32_t* seq_lens, int32_t B, int32_t max_seq_len, void* out, void* workspace,
                             size_t workspace_bytes, void* stream) {
  g4_status st = kv4_check_params(params);
  if (st != G4_OK) return st;
  if (B < 0) return fail(G4_ERR_INVALID_ARG, "B %d must be >= 0", B);
  if (q == nullptr || out == nullptr || seq_lens == nullptr)
    return fail(G4_ERR_INVALID_ARG, "q, out and seq_lens must be non-NULL");
  if (!aligned16(q) || !aligned16(out)) return fail(G4_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  const g4_kv4_pool* c = nullptr;
  st = kv4_resolve_src(params, pools, n_layers, layer, &c);
  if (st != G4_OK) return st;
  st = kv4_check_table(block_table, max_blocks, c->block_size);
  if (st != G4_OK) return st;
  if (max_seq_len < 1 || max_seq_len > max_blocks * c->block_size)
    return fail(G4_ERR_CAPACITY, "max_seq_len %d outside [1, %d blocks of %d]", max_seq_len, max_blocks, c->block_size);
  if (B == 0) return ok();
  const int window = params->layer_type == G4_SLIDING ? params->window : 0;
  const g4::Kv4DecodePlan plan =
      g4::kv4_decode_plan(window, params->head_dim, params->n_heads, params->n_kv_heads, B, max_seq_len);
  // A CTA counts its share's records in 32 bits.
  const long long span = window > 0 && window < max_seq_len ? window : max_seq_len;
  if (static_cast<long long>(B) * params->n_kv_heads > 0x7fffff00LL / (span / 16 + 2) * plan.nctas)
    return fail(G4_ERR_UNSUPPORTED, "%d sequences of %lld keys are more than a call can count", B, span);
  if (workspace_bytes < plan.ws_bytes)
    return fail(G4_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed", workspace_bytes, plan.ws_bytes);
  if (plan.ws_bytes > 0 && (workspace == nullptr || !aligned16(workspace)))
    return fail(G4_ERR_INVALID_ARG, "workspace must be non-NULL and 16-byte aligned");
  int* err = device_error_ptr();
  if (err == nullptr) return fail(G4_ERR_CUDA, "cannot resolve the device error word");
  g4::Kv4DecodeArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.data = static_cast<const uint8_t*>(c->data);
  a.table = block_table;
  a.lens = seq_lens;
  a.out = out;
  a.err = err;
  a.B = B;
  a.H = params->n_heads;
  a.Hkv = params->n_kv_heads;
  a.hd = params->head_dim;
  a.max_blocks = max_blocks;
  a.n_blocks = c->n_blocks;
  a.block_shift = log2_of(c->block_size);
  a.window = window;
  a.len_cap = max_seq_len;
  a.nctas = plan.nctas;
  a.scale_log2 = params->attn_scale * 1.4426950408889634f * static_cast<float>(ldexp(1.0, c->k_exp));
  if (plan.ws_bytes > 0) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.tickets = reinterpret_cast<unsigned*>(ws);
    a.ws_ml = reinterpret_cast<float2*>(ws + g4::kKv4TicketBytes);
    a.ws_o = reinterpret_cast<float*>(ws + g4::kKv4TicketBytes + plan.ml_bytes);
  }
  return cuda_status(g4::launch_kv4_decode(a, static_cast<cudaStream_t>(stream)), "4-bit decode launch");
}

size_t g4_kv4_prefill_workspace_size(const g4_layer_params* params, int32_t B, int32_t T, int32_t max_seq_len) {
  if (kv4_check_params(params) != G4_OK || B < 1 || T < 1 || max_seq_len < T || max_seq_len > 0x7fffffff - T) return 0;
  return kv4_prefill_head_bytes(B) + 2 * kv4_prefill_kv_bytes(params, B, T, max_seq_len);
}

g4_status g4_kv4_attn_prefill(const g4_layer_params* params, const g4_kv4_pool* pools, int32_t n_layers,
                              int32_t layer, const void* q, const int32_t* block_table, int32_t max_blocks,
                              const int32_t* q_start_pos, const int32_t* seq_lens, int32_t B, int32_t T,
                              int32_t max_seq_len, void* out, void* workspace, size_t workspace_bytes,
                              void* stream) {
  g4_status st = kv4_check_params(params);
  if (st != G4_OK) return st;
  if (B < 0 || T < 0) return fail(G4_ERR_INVALID_ARG, "B %d and T %d must be >= 0", B, T);
  if (q == nullptr || out == nullptr || q_start_pos == nullptr || seq_lens == nullptr)
    return fail(G4_ERR_INVALID_ARG, "q, out, q_start_pos and seq_lens must be non-NULL");
  if (!aligned16(q) || !aligned16(out)) return fail(G4_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  const g4_kv4_pool* c = nullptr;
  st = kv4_resolve_src(params, pools, n_layers, layer, &c);
  if (st != G4_OK) return st;
  st = kv4_check_table(block_table, max_blocks, c->block_size);
  if (st != G4_OK) return st;
  if (max_seq_len < 1 || max_seq_len > max_blocks * c->block_size)
    return fail(G4_ERR_CAPACITY, "max_seq_len %d outside [1, %d blocks of %d]", max_seq_len, max_blocks, c->block_size);
  if (T > max_seq_len || max_seq_len > 0x7fffffff - T)
    return fail(G4_ERR_CAPACITY, "T %d exceeds max_seq_len %d, or both together 2^31 - 1", T, max_seq_len);
  if (B == 0 || T == 0) return ok();
  const size_t head = kv4_prefill_head_bytes(B), kv = kv4_prefill_kv_bytes(params, B, T, max_seq_len);
  if (workspace_bytes < head + 2 * kv)
    return fail(G4_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed", workspace_bytes, head + 2 * kv);
  if (workspace == nullptr || !aligned16(workspace))
    return fail(G4_ERR_INVALID_ARG, "workspace must be non-NULL and 16-byte aligned");
  int* err = device_error_ptr();
  if (err == nullptr) return fail(G4_ERR_CUDA, "cannot resolve the device error word");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Two launches: a key is read by every query tile of every head of its group, so
  // it is widened once, into the rows that the tensor-core prefill loads by TMA.  The
  // gather is 14 us of 203 at 2 x 2048 tokens of 8 heads of 512 (full layer), 4 of 20
  // at 4 x 256 tokens of a sliding layer.
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  g4::Kv4GatherArgs ga;
  memset(&ga, 0, sizeof(ga));
  ga.data = static_cast<const uint8_t*>(c->data);
  ga.table = block_table;
  ga.lens = seq_lens;
  ga.q_start = q_start_pos;
  ga.q_rel = reinterpret_cast<int32_t*>(ws);
  ga.k = ws + head;
  ga.v = ws + head + kv;
  ga.B = B;
  ga.Hkv = params->n_kv_heads;
  ga.hd = params->head_dim;
  ga.rows = kv4_prefill_rows(params, T, max_seq_len);
  ga.max_blocks = max_blocks;
  ga.n_blocks = c->n_blocks;
  ga.block_shift = log2_of(c->block_size);
  ga.T = T;
  ga.window = params->layer_type == G4_SLIDING ? params->window : 0;
  ga.max_seq_len = max_seq_len;
  ga.k_mul = static_cast<float>(ldexp(1.0, c->k_exp));
  st = cuda_status(g4::launch_kv4_gather(ga, s), "4-bit prefill's gather launch");
  if (st != G4_OK) return st;
  g4::PrefillTcArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.ck = ga.k;
  a.cv = ga.v;
  a.out = out;
  a.q_start = ga.q_rel;
  a.err = err;
  a.B = B;
  a.T = T;
  a.H = params->n_heads;
  a.Hkv = params->n_kv_heads;
  a.hd = params->head_dim;
  a.max_len = ga.rows;
  a.sliding = params->layer_type == G4_SLIDING;
  a.window = params->window;
  a.scale_log2 = params->attn_scale * 1.4426950408889634f;
  return cuda_status(g4::launch_prefill_tc(a, s), "tcgen05 prefill launch");
}

}  // extern "C"

namespace {

// The mods of a call, checked against the layer; *m is `given` or, for none, all zeros.
g4_status check_mods(const g4_layer_params* p, const g4_score_mods* given, g4_score_mods* m) {
  memset(m, 0, sizeof(*m));
  if (given == nullptr) return G4_OK;
  *m = *given;
  if (m->softcap != 0.0f && !(m->softcap >= 0x1.0p-10f && m->softcap <= 0x1.0p10f))
    return fail(G4_ERR_UNSUPPORTED, "softcap %g is neither 0 nor in [2^-10, 2^10]", static_cast<double>(m->softcap));
  if (!aligned4(m->slopes) || !aligned4(m->key_begin) || !aligned4(m->key_end))
    return fail(G4_ERR_INVALID_ARG, "slopes, key_begin and key_end must be 4-byte aligned");
  if (m->softcap != 0.0f && !isfinite(p->attn_scale * 2.8853900817779268f / m->softcap))
    return fail(G4_ERR_UNSUPPORTED, "attn_scale %g is too large for softcap %g", static_cast<double>(p->attn_scale),
                static_cast<double>(m->softcap));
  return G4_OK;
}

}  // namespace

extern "C" {

g4_status g4_attn_visible_ranges(int32_t window, const int32_t* q_start_pos, const int32_t* seq_lens,
                                 const int32_t* doc_ids, const int32_t* span_ids, int32_t max_len, int32_t B, int32_t T,
                                 int32_t* key_begin, int32_t* key_end, void* stream) {
  if (B < 0 || T < 0 || window < 0) return fail(G4_ERR_INVALID_ARG, "B %d, T %d and window %d must be >= 0", B, T, window);
  if (max_len < 1) return fail(G4_ERR_INVALID_ARG, "max_len %d must be >= 1", max_len);
  if (max_len > 1 << 24) return fail(G4_ERR_UNSUPPORTED, "max_len %d exceeds 2^24", max_len);
  if (B > 1 << 20) return fail(G4_ERR_UNSUPPORTED, "B %d exceeds 2^20", B);
  if (static_cast<long long>(B) * T > 0x7fffffffLL) return fail(G4_ERR_INVALID_ARG, "B * T exceeds 2^31 - 1");
  if (q_start_pos == nullptr || seq_lens == nullptr || key_begin == nullptr || key_end == nullptr)
    return fail(G4_ERR_INVALID_ARG, "q_start_pos, seq_lens, key_begin and key_end must be non-NULL");
  if (!aligned4(q_start_pos) || !aligned4(seq_lens) || !aligned4(doc_ids) || !aligned4(span_ids) || !aligned4(key_begin) ||
      !aligned4(key_end))
    return fail(G4_ERR_INVALID_ARG, "positions, lengths, ids and intervals must be 4-byte aligned");
  if (B == 0 || T == 0) return ok();
  g4::RangesArgs a;
  memset(&a, 0, sizeof(a));
  a.q_start = q_start_pos;
  a.lens = seq_lens;
  a.doc = doc_ids;
  a.span = span_ids;
  a.begin = key_begin;
  a.end = key_end;
  a.B = B;
  a.T = T;
  a.max_len = max_len;
  a.window = window;
  return cuda_status(g4::launch_ranges(a, static_cast<cudaStream_t>(stream)), "visible ranges launch");
}

g4_status g4_kv_append_normrope_axes(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                                     int32_t layer, const g4_rope_axes* axes, const void* q_in, const void* k_in,
                                     const void* v_in, const float* q_norm_w, const float* k_norm_w,
                                     const int32_t* positions, const int32_t* rows, int32_t B, int32_t T, void* q_out,
                                     void* stream) {
  g4_status st = check_params(params);
  if (st != G4_OK) return st;
  if (B < 0 || T < 0) return fail(G4_ERR_INVALID_ARG, "B %d and T %d must be >= 0", B, T);
  if (axes == nullptr || axes->axis == nullptr) return fail(G4_ERR_INVALID_ARG, "axes and their table must be non-NULL");
  if (axes->n_axes < 1 || axes->n_axes > 4)
    return fail(G4_ERR_UNSUPPORTED, "%d axes not supported (1 to 4)", axes->n_axes);
  if (q_in == nullptr || q_out == nullptr || q_norm_w == nullptr || positions == nullptr)
    return fail(G4_ERR_INVALID_ARG, "q_in, q_out, q_norm_w and positions must be non-NULL");
  if (!aligned16(q_in) || !aligned16(q_out) || !aligned16(q_norm_w))
    return fail(G4_ERR_INVALID_ARG, "q_in, q_out and q_norm_w must be 16-byte aligned");
  if (!aligned4(positions) || !aligned4(rows)) return fail(G4_ERR_INVALID_ARG, "positions and rows must be 4-byte aligned");
  const bool shared = params->kv_share_src >= 0;
  g4::AxesAppendArgs a;
  memset(&a, 0, sizeof(a));
  if (shared) {
    if (k_in != nullptr || v_in != nullptr || k_norm_w != nullptr)
      return fail(G4_ERR_INVALID_ARG, "layer %d shares the cache of layer %d: k_in, v_in and k_norm_w must be NULL",
                  layer, params->kv_share_src);
    if (layer < 0 || layer >= n_layers) return fail(G4_ERR_INVALID_ARG, "layer %d outside [0, %d)", layer, n_layers);
  } else {
    if (k_in == nullptr || v_in == nullptr || k_norm_w == nullptr || rows == nullptr)
      return fail(G4_ERR_INVALID_ARG, "layer %d owns its cache: k_in, v_in, k_norm_w and rows must be non-NULL", layer);
    if (!aligned16(k_in) || !aligned16(v_in) || !aligned16(k_norm_w))
      return fail(G4_ERR_INVALID_ARG, "k_in, v_in and k_norm_w must be 16-byte aligned");
    const g4_kv_cache* c = nullptr;
    st = resolve_src(params, caches, n_layers, layer, &c);
    if (st != G4_OK) return st;
    if (c->batch < B) return fail(G4_ERR_CAPACITY, "cache batch %d < B %d", c->batch, B);
    a.cache_k = c->k;
    a.cache_v = c->v;
    a.max_len = c->max_len;
    a.ring = c->ring;
    a.k_in = k_in;
    a.v_in = v_in;
    a.k_w = k_norm_w;
    a.rows = rows;
  }
  const long long tokens = static_cast<long long>(B) * T;
  if (tokens > 0x7fffffffLL) return fail(G4_ERR_INVALID_ARG, "B * T exceeds 2^31 - 1");
  rope_table(params, &a.n_rot, a.inv_freq);
  for (int j = 0; j < a.n_rot; ++j) {
    if (axes->axis[j] >= axes->n_axes)
      return fail(G4_ERR_INVALID_ARG, "pair %d is turned by axis %d of %d", j, axes->axis[j], axes->n_axes);
    a.axis[j] = axes->axis[j];
    if (axes->inv_freq != nullptr) {
      if (!(axes->inv_freq[j] >= 0.0f && axes->inv_freq[j] <= 1.0f))
        return fail(G4_ERR_INVALID_ARG, "inv_freq of pair %d outside [0, 1]", j);
      a.inv_freq[j] = axes->inv_freq[j];
    }
  }
  if (tokens == 0) return ok();
  a.n_axes = axes->n_axes;
  a.q_in = q_in;
  a.q_w = q_norm_w;
  a.positions = positions;
  a.q_out = q_out;
  a.B = B;
  a.T = T;
  a.H = params->n_heads;
  a.Hkv = params->n_kv_heads;
  a.hd = params->head_dim;
  a.eps = params->eps;
  a.err = device_error_ptr();
  if (a.err == nullptr) return fail(G4_ERR_CUDA, "cannot resolve the device error word");
  // A warp takes a token's rows as long as that makes 16 warps for each SM, fewer of them otherwise.
  const int nrows = a.H + (shared ? 0 : 2 * a.Hkv);
  const long long rows_each = tokens * nrows / (16LL * g4::sm_count());
  a.rows_per_unit = static_cast<int>(rows_each < 1 ? 1 : rows_each > nrows ? nrows : rows_each);
  return cuda_status(g4::launch_append_axes(a, params->dtype, static_cast<cudaStream_t>(stream)), "append launch");
}

g4_status g4_attn_prefill_mods(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                               int32_t layer, const g4_score_mods* mods, const void* q, const int32_t* q_start_pos,
                               int32_t B, int32_t T, void* out, void* stream) {
  g4_status st = check_params(params);
  if (st != G4_OK) return st;
  if (B < 0 || T < 0) return fail(G4_ERR_INVALID_ARG, "B %d and T %d must be >= 0", B, T);
  if (q == nullptr || out == nullptr || q_start_pos == nullptr)
    return fail(G4_ERR_INVALID_ARG, "q, out and q_start_pos must be non-NULL");
  if (!aligned16(q) || !aligned16(out)) return fail(G4_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if (!aligned4(q_start_pos)) return fail(G4_ERR_INVALID_ARG, "q_start_pos must be 4-byte aligned");
  g4_score_mods m;
  st = check_mods(params, mods, &m);
  if (st != G4_OK) return st;
  const g4_kv_cache* c = nullptr;
  st = resolve_src(params, caches, n_layers, layer, &c);
  if (st != G4_OK) return st;
  if (c->batch < B) return fail(G4_ERR_CAPACITY, "cache batch %d < B %d", c->batch, B);
  if (c->ring) {
    // As in g4_attn_prefill; intervals of the caller's own may begin where they like.
    if (T > c->max_len || (m.key_begin == nullptr && static_cast<long long>(T) + params->window - 1 > c->max_len))
      return fail(G4_ERR_CAPACITY, "ring cache of %d rows cannot hold the %d + %d - 1 keys a chunk of T = %d needs",
                  c->max_len, T, params->window, T);
    if (params->dtype == G4_BF16 && c->max_len % 128 != 0)
      return fail(G4_ERR_UNSUPPORTED, "bf16 prefill on a ring cache needs max_len a multiple of 128 (got %d)",
                  c->max_len);
  } else if (T > c->max_len) {
    return fail(G4_ERR_CAPACITY, "T %d exceeds the cache length %d", T, c->max_len);
  }
  if (B == 0 || T == 0) return ok();
  int* err = device_error_ptr();
  if (err == nullptr) return fail(G4_ERR_CUDA, "cannot resolve the device error word");
  const float scale_log2 = params->attn_scale * 1.4426950408889634f;
  const float cap_log2 = m.softcap * 1.4426950408889634f;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (params->dtype == G4_BF16) {
    g4::ModsTcArgs a;
    memset(&a, 0, sizeof(a));
    a.q = q;
    a.ck = c->k;
    a.cv = c->v;
    a.out = out;
    a.q_start = q_start_pos;
    a.err = err;
    a.B = B;
    a.T = T;
    a.H = params->n_heads;
    a.Hkv = params->n_kv_heads;
    a.hd = params->head_dim;
    a.max_len = c->max_len;
    a.ring = c->ring;
    a.sliding = params->layer_type == G4_SLIDING;
    a.window = params->window;
    a.scale_log2 = scale_log2;
    a.cap_log2 = cap_log2;
    a.cap_in = m.softcap != 0.0f ? 2.0f * scale_log2 / m.softcap : 0.0f;
    a.slopes = m.slopes;
    a.key_begin = m.key_begin;
    a.key_end = m.key_end;
    return cuda_status(g4::launch_prefill_mods(a, s), "tcgen05 prefill launch");
  }
  g4::ModsSimtArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.ck = c->k;
  a.cv = c->v;
  a.out = out;
  a.base = q_start_pos;
  a.err = err;
  a.mode = 1;
  a.B = B;
  a.T = T;
  a.H = params->n_heads;
  a.Hkv = params->n_kv_heads;
  a.hd = params->head_dim;
  a.max_len = c->max_len;
  a.ring = c->ring;
  a.sliding = params->layer_type == G4_SLIDING;
  a.window = params->window;
  a.len_cap = c->max_len;
  a.chunk = c->max_len;  // one split holds any interval
  a.nsplit = 1;
  a.scale_log2 = scale_log2;
  a.cap_log2 = cap_log2;
  a.slopes = m.slopes;
  a.key_begin = m.key_begin;
  a.key_end = m.key_end;
  return cuda_status(g4::launch_attn_simt_mods(a, s), "float32 prefill launch");
}

size_t g4_attn_decode_mods_workspace_size(const g4_layer_params* params, int32_t B, int32_t max_seq_len) {
  if (check_params(params) != G4_OK || B < 1 || max_seq_len < 1) return 0;
  return g4::mods_decode_plan(params->dtype, params->layer_type == G4_SLIDING ? params->window : 0, params->head_dim,
                              params->n_heads, params->n_kv_heads, B, max_seq_len)
      .ws_bytes;
}

g4_status g4_attn_decode_mods(const g4_layer_params* params, const g4_kv_cache* caches, int32_t n_layers,
                              int32_t layer, const g4_score_mods* mods, const void* q, const int32_t* seq_lens,
                              int32_t B, int32_t max_seq_len, void* out, void* workspace, size_t workspace_bytes,
                              void* stream) {
  g4_status st = check_params(params);
  if (st != G4_OK) return st;
  if (B < 0) return fail(G4_ERR_INVALID_ARG, "B %d must be >= 0", B);
  if (q == nullptr || out == nullptr || seq_lens == nullptr)
    return fail(G4_ERR_INVALID_ARG, "q, out and seq_lens must be non-NULL");
  if (!aligned16(q) || !aligned16(out)) return fail(G4_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if (!aligned4(seq_lens)) return fail(G4_ERR_INVALID_ARG, "seq_lens must be 4-byte aligned");
  g4_score_mods m;
  st = check_mods(params, mods, &m);
  if (st != G4_OK) return st;
  if (m.key_end != nullptr) return fail(G4_ERR_INVALID_ARG, "the new token is its sequence's last key: key_end must be NULL");
  const g4_kv_cache* c = nullptr;
  st = resolve_src(params, caches, n_layers, layer, &c);
  if (st != G4_OK) return st;
  if (c->batch < B) return fail(G4_ERR_CAPACITY, "cache batch %d < B %d", c->batch, B);
  if (max_seq_len < 1 || (!c->ring && max_seq_len > c->max_len))
    return fail(G4_ERR_CAPACITY, "max_seq_len %d outside [1, cache length %d]", max_seq_len, c->max_len);
  if (B == 0) return ok();
  const int window = params->layer_type == G4_SLIDING ? params->window : 0;
  const g4::ModsDecodePlan plan = g4::mods_decode_plan(params->dtype, window, params->head_dim, params->n_heads,
                                                       params->n_kv_heads, B, max_seq_len);
  if (workspace_bytes < plan.ws_bytes)
    return fail(G4_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed", workspace_bytes, plan.ws_bytes);
  if (plan.ws_bytes > 0 && (workspace == nullptr || !aligned16(workspace)))
    return fail(G4_ERR_INVALID_ARG, "workspace must be non-NULL and 16-byte aligned");
  int* err = device_error_ptr();
  if (err == nullptr) return fail(G4_ERR_CUDA, "cannot resolve the device error word");
  const float scale_log2 = params->attn_scale * 1.4426950408889634f;
  const float cap_log2 = m.softcap * 1.4426950408889634f;
  if (plan.win) {
    g4::ModsWinArgs w;
    memset(&w, 0, sizeof(w));
    w.q = q;
    w.ck = c->k;
    w.cv = c->v;
    w.out = out;
    w.base = seq_lens;
    w.err = err;
    w.B = B;
    w.T = 1;
    w.H = params->n_heads;
    w.Hkv = params->n_kv_heads;
    w.hd = params->head_dim;
    w.max_len = c->max_len;
    w.ring = c->ring;
    w.sliding = window > 0;
    w.window = window;
    w.len_cap = max_seq_len;
    w.chunk = 64;
    w.nsplit = g4::decode_win_splits(window > 0 && window < max_seq_len ? window : max_seq_len);
    w.scale_log2 = scale_log2;
    w.cap_log2 = cap_log2;
    w.slopes = m.slopes;
    w.key_begin = m.key_begin;
    return cuda_status(g4::launch_decode_win_mods(w, static_cast<cudaStream_t>(stream)), "windowed decode launch");
  }
  g4::ModsDecodeArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.ck = c->k;
  a.cv = c->v;
  a.out = out;
  a.lens = seq_lens;
  a.key_begin = m.key_begin;
  a.slopes = m.slopes;
  a.err = err;
  a.B = B;
  a.H = params->n_heads;
  a.Hkv = params->n_kv_heads;
  a.hd = params->head_dim;
  a.max_len = c->max_len;
  a.ring = c->ring;
  a.window = window;
  a.len_cap = max_seq_len;
  a.nctas = plan.nctas;
  a.scale_log2 = scale_log2;
  a.cap_log2 = cap_log2;
  if (plan.ws_bytes > 0) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.tickets = reinterpret_cast<unsigned*>(ws);
    a.ws_ml = reinterpret_cast<float2*>(ws + plan.t_bytes);
    a.ws_o = reinterpret_cast<float*>(ws + plan.t_bytes + plan.ml_bytes);
  }
  return cuda_status(g4::launch_decode_mods(a, params->dtype, plan.warps, static_cast<cudaStream_t>(stream)),
                     "decode launch");
}

const char* g4_last_error(void) { return g_last_error.c_str(); }

int32_t g4_take_device_error(void) {
  int* p = device_error_ptr();
  if (p == nullptr) return -1;
  int v = 0;
  if (cudaDeviceSynchronize() != cudaSuccess) return -1;
  if (cudaMemcpy(&v, p, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return -1;
  const int zero = 0;
  if (cudaMemcpy(p, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return -1;
  return v;
}

}  // extern "C"
