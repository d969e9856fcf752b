// Internal launch interface of the paged 4-bit cache between the C-ABI front
// end (g4_api.cu) and its kernels (g4_append.cu, g4_kv4_cache.cu,
// g4_kv4_decode.cu).  The cache's layout: include/g4attn.h and g4_kv4.cuh.
#pragma once

#include "g4_internal.h"

namespace g4 {

struct Kv4AssignArgs {
  int B, T, block_shift, n_blocks, max_blocks;
  const int32_t* old_lens;
  const int32_t* new_lens;
  int32_t* free_blocks;
  const int32_t* free_count;
  int32_t* table;
  int32_t* lens_out;
  int32_t* count_out;
  int32_t* positions;
  int32_t* slots;
};
constexpr int kKv4MaxBatch = 8192;  // a CTA keeps 8 to 16 bytes per sequence in shared memory
cudaError_t launch_kv4_assign(const Kv4AssignArgs& a, cudaStream_t s);

// The append into a pool.  cache_k is the layer's pool; tok_per_cta at most kAppendMaxTokens.
constexpr int kAppendMaxTokens = 4;
struct Kv4AppendArgs : AppendArgs {
  const int32_t* slots;  // [B*T]
  int n_slots;           // n_blocks * block_size
  int block_shift;       // log2(block_size)
  float k_mul;           // 2^-k_exp
};
cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t s);

// Positions [first, first + rows) of every sequence as bf16 rows
// k, v [B][Hkv][rows][hd].  first is start[b], or with q_start set (prefill)
// the first position that any of T queries from q_start[b] on sees; then only
// rows up to the last query are written, and q_rel[b] is the first query's row.
struct Kv4GatherArgs {
  const uint8_t* data;
  const int32_t* table;
  const int32_t* start;
  const int32_t* lens;
  const int32_t* q_start;
  int32_t* q_rel;
  void* k;
  void* v;
  int B, Hkv, hd, rows, max_blocks, n_blocks, block_shift;
  int T, window, max_seq_len;  // prefill; window 0 on a full layer
  float k_mul;                 // 2^k_exp
  int per_unit;                // CTAs per sequence and kv head (set by the launch)
};
cudaError_t launch_kv4_gather(const Kv4GatherArgs& a, cudaStream_t s);

struct Kv4DecodeArgs {
  const void* q;  // [B][H][hd] bf16
  const uint8_t* data;
  const int32_t* table;
  const int32_t* lens;
  void* out;
  float* ws_o;        // [2 nctas][G][hd] partial outputs: two units of a CTA's share may continue in other CTAs'
  float2* ws_ml;      // [2 nctas][8] their softmax references and denominators
  unsigned* tickets;  // arrival counters (zero between calls), [4 levels of merges][2 kKv4MaxCtas]
  int* err;
  int B, H, Hkv, hd, max_blocks, n_blocks, block_shift;
  int window;  // 0 on a full layer
  int len_cap;
  int nctas;
  float scale_log2;  // attn_scale * log2(e) * 2^k_exp
};
// Workspace: the tickets, then ws_ml, then ws_o.  The tickets are in front and of
// a fixed size, so calls of different shapes may take turns on one workspace.
constexpr int kKv4MaxCtas = 1024;
constexpr size_t kKv4TicketBytes = 4 * 2 * kKv4MaxCtas * 4;
struct Kv4DecodePlan {
  int nctas;
  size_t ml_bytes, o_bytes, ws_bytes;
};
Kv4DecodePlan kv4_decode_plan(int window, int hd, int H, int Hkv, int B, int max_seq_len);
cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, cudaStream_t s);

}  // namespace g4
