// Step a4: fused per-head RMSNorm -> rotate_half RoPE -> KV-cache append.
//
// cortiq-engine g4e.rs `g4e_forward` (attention block): q heads are normed
// with q_norm and roped; on a layer that owns its cache, k heads are normed
// with k_norm and roped, v heads get the weight-less norm (`rms_plain`), and
// both are appended at the token's position.  ferrox-models
// gemma4_engine.rs `forward_token_on_worker` does the same per head
// (`rms_norm_per_head`, `apply_rope`, `cache.push`).  turbospark-runtime
// gemma4/attn.rs writes the projections straight into the cache slot and
// norms/ropes them there, which is the fusion done here.  A token at
// position p goes to cache row p, or p mod max_len on a sliding-window ring.
//
// One CTA (4 warps) handles the tokens at one t of up to tok_per_cta
// consecutive sequences, rows_per_cta of each token's H + 2*Hkv head rows;
// one warp per head row.  The cos/sin table (head_dim / 2 pairs,
// double-float) is built per distinct position from angle = pos *
// inv_freq[j] with inv_freq a float32 table.  Pairs j >= n_rot (zero inv_freq) are left
// unrotated, so those dims are the normed input.  bf16 stores are the
// correctly rounded real results (g4_normrope.cuh), decided in three stages:
//   1. float32 for the whole row (packed float32x2 products), with Ziv's test
//      of each value against its error bound; in the synthetic workloads
//      about one row in five has a value the test leaves open;
//   2. for those values only, lane by lane: the float32 inverse rms times the
//      row's inner products in double-float, whose error is the inverse
//      rms's alone; this leaves open about one row in twenty to thirty;
//   3. the row's sum of squares in double-float (error-free splitting) and a
//      double-float inverse rms, which decide the rest.
//
// The 4-bit cache's append (KV4) differs in where rows go: a row is finished in
// shared memory, then a q row is copied out and a k or v row quantised by
// kv4_store_row; all tokens' cos/sin tables are built at once.  Bound by
// instruction issue (2.7 per cycle): 8 sequences x 2048 tokens of 8 + 2 + 2 rows
// of 512 take 155 us where the sequences' positions differ, 138 where they agree (the bf16
// append: 179 and 114), 59 us of which are bytes; with the stores left out 2 %
// less.
//
// Lane l of a warp owns elements [l*E, l*E + E) of the lower half and the
// same offsets of the upper half (E = head_dim / 64), so each rotate_half
// pair (j, j + head_dim/2) sits in one lane.  Each warp loads its next row
// before it computes the current one.
//
// q_out = q_in (IN_PLACE, bf16): stages 2 and 3 look at a row's elements again,
// which stage 1 has overwritten by then, so lanes with open values keep theirs in
// shared memory: 8 x 2048 tokens of 8 + 2 + 2 rows of 512 119 us (apart 111), of 256 75 (74), of 128 49
// (52); with the kernel of several axes, 121, 102 and 69.  Four CTAs per SM at 512, since at five the next
// row's elements are spilled, and so waited for, as soon as they are asked for: 285 us.
#include <type_traits>

#include "g4_device.cuh"
#include "g4_internal.h"
#include "g4_kv4.cuh"
#include "g4_kv4_internal.h"
#include "g4_normrope.cuh"

namespace g4 {
namespace {

// The bits of a lane's E consecutive elements of one half of a head row.
template <typename T, int E>
struct HalfBits;
template <int E>
struct HalfBits<float, E> {
  float v[E];
};
template <int E>
struct HalfBits<__nv_bfloat16, E> {
  uint32_t v[(E + 1) / 2];
};

template <int E>
__device__ __forceinline__ void load_bits(const float* p, HalfBits<float, E>& h) {
  load_elems<E>(p, h.v);
}
template <int E>
__device__ __forceinline__ void load_bits(const __nv_bfloat16* p, HalfBits<__nv_bfloat16, E>& h) {
  if constexpr (E == 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    h.v[0] = v.x; h.v[1] = v.y; h.v[2] = v.z; h.v[3] = v.w;
  } else if constexpr (E == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    h.v[0] = v.x; h.v[1] = v.y;
  } else if constexpr (E == 2) {
    h.v[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    h.v[0] = *reinterpret_cast<const uint16_t*>(p);
  }
}

template <int E>
__device__ __forceinline__ void store_bits(__nv_bfloat16* p, const HalfBits<__nv_bfloat16, E>& h) {
  if constexpr (E == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(h.v[0], h.v[1], h.v[2], h.v[3]);
  } else if constexpr (E == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(h.v[0], h.v[1]);
  } else if constexpr (E == 2) {
    *reinterpret_cast<uint32_t*>(p) = h.v[0];
  } else {
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(h.v[0]);
  }
}

template <int E>
__device__ __forceinline__ void unpack_bits(const HalfBits<float, E>& h, float* x) {
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = h.v[i];
}
template <int E>
__device__ __forceinline__ void unpack_bits(const HalfBits<__nv_bfloat16, E>& h, float* x) {
  if constexpr (E == 1) {
    x[0] = bf16_lo(h.v[0]);
  } else {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      x[2 * i] = bf16_lo(h.v[i]);
      x[2 * i + 1] = bf16_hi(h.v[i]);
    }
  }
}

// y = (x * r) * w elementwise (w == nullptr: y = x * r), two elements per
// packed float32x2 instruction; each product is rounded as its own float op.
template <int E>
__device__ __forceinline__ void scale_elems(float* y, const float* x, float r, const float* w) {
  if constexpr (E % 2 == 0) {
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      float2 t = __fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(r, r));
      if (w != nullptr) t = __fmul2_rn(t, make_float2(w[i], w[i + 1]));
      y[i] = t.x;
      y[i + 1] = t.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) y[i] = w != nullptr ? (x[i] * r) * w[i] : x[i] * r;
  }
}

// rotate_half on the lane's pairs: oa = ya c - yb s, ob = yb c + ya s, each
// as one fma over one rounded product.
template <int E>
__device__ __forceinline__ void rotate_elems(float* oa, float* ob, const float* ya, const float* yb, const float* c,
                                             const float* s) {
  if constexpr (E % 2 == 0) {
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 a2 = make_float2(ya[i], ya[i + 1]);
      const float2 b2 = make_float2(yb[i], yb[i + 1]);
      const float2 c2 = make_float2(c[i], c[i + 1]);
      const float2 ra = __ffma2_rn(a2, c2, __fmul2_rn(b2, make_float2(-s[i], -s[i + 1])));
      const float2 rb = __ffma2_rn(b2, c2, __fmul2_rn(a2, make_float2(s[i], s[i + 1])));
      oa[i] = ra.x; oa[i + 1] = ra.y;
      ob[i] = rb.x; ob[i + 1] = rb.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      oa[i] = fmaf(ya[i], c[i], yb[i] * -s[i]);
      ob[i] = fmaf(yb[i], c[i], ya[i] * s[i]);
    }
  }
}

// True when no bf16 rounding boundary lies within e of v (so v's own bf16
// rounding is that of every value within e of it).
__device__ __forceinline__ bool bf16_decided(float v, float e) { return fabsf(v - bf16_midpoint(v)) > e; }

// Where element d of a finished row lies: 64-element pieces are 16 bytes apart,
// so that the 16-byte halves of neighbouring lanes' 32 bytes meet other banks.
__host__ __device__ constexpr int kv4_row_at(int d) { return d + (d >> 6) * 8; }

// Quantises a finished row (bf16 values in shared memory, by kv4_row_at) and
// stores codes and scales of position m into its record.  Lane l takes the
// HD / 32 elements from l HD / 32 on: a whole block of 16, or a part of one whose
// other lanes it asks for the largest magnitude.  The code bytes of the 4
// blocks that the record keeps side by side are then exchanged between their
// lanes, so that each lane has bytes that lie together.
//   The divisions x / s and max / 6 are products with a rounded reciprocal,
// brought back by a rounding to 2^-12 (x / s: at most 12 where s did not saturate
// at 448, and past that the code saturates too) or to 16
// significant bits (max / 6).  That is as good as the exact quotient: x and max
// have 8 significant bits, the numbers between which codes and scales change, times s
// or 6, at most 7 (3 of a code times 4 of a scale; 5 of a scale times 2 of a 6), so
// a quotient is one of those numbers or at least 2^-8 (relative) away, where the
// products are off by 2^-22.
template <int HD>
__device__ __forceinline__ void kv4_store_row(const __nv_bfloat16* row, uint8_t* rec, int m, bool is_k, float mul,
                                              int lane) {
  constexpr int N = HD / 32;       // elements of this lane
  constexpr int LPB = 16 / N;      // lanes per block
  constexpr unsigned kAll = 0xffffffffu;
  const int d0 = lane * N;
  uint32_t w[N / 2];               // bf16 pairs
  const uint32_t* src = reinterpret_cast<const uint32_t*>(row + kv4_row_at(d0));
  if constexpr (N >= 8) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(src)[i];
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = src[i];
  }
  // largest magnitude, as bits (NaN > infinity > the rest): 16-bit halves compare as integers
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
  top = max(top & 0xffffu, top >> 16);
#pragma unroll
  for (int o = 1; o < LPB; o <<= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
  const bool finite = top < 0x7f80u;
  const float q6 = __uint_as_float(top << 16) * mul * (1.0f / 6.0f);
  const uint32_t byte = finite ? e4m3_byte(__uint_as_float((__float_as_uint(q6) + 0x80u) & ~0xffu)) : 0x7fu;
  const float s = e4m3_value(byte);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  const bool coded = s > 0.0f;  // else a block of zeros (or all too small), or one that holds a NaN or an infinity: codes 0
  inv = coded ? inv * mul : 0.0f;
  uint32_t code[(N + 7) / 8] = {};    // code bytes, in order
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    constexpr float kSnap = 0x1.8p11f;  // adding it rounds to a multiple of 2^-12
    const float2 x = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
    float2 q = __fmul2_rn(x, make_float2(inv, inv));
    q = __fadd2_rn(__fadd2_rn(q, make_float2(kSnap, kSnap)), make_float2(-kSnap, -kSnap));
    // (a quotient that rounds to zero keeps its sign)
    code[i / 4] |= e2m1x2_byte(__uint_as_float(__float_as_uint(q.x) | (__float_as_uint(x.x) & 0x80000000u)),
                               __uint_as_float(__float_as_uint(q.y) | (__float_as_uint(x.y) & 0x80000000u)))
                   << (8 * (i % 4));
  }
#pragma unroll
  for (int i = 0; i < (N + 7) / 8; ++i) code[i] = coded ? code[i] : 0u;  // (a NaN's would be 6's)
  if (lane % LPB == 0)
    rec[is_k ? kv4_k_scale_at<HD>(m, d0) : kv4_v_scale_at<HD>(m, d0)] = static_cast<uint8_t>(byte);

  const int blk = lane / LPB, p0 = blk / 4 * 64;  // its piece begins at element p0
  if constexpr (HD >= 256) {
    // the four blocks of a piece are lanes blk % 4 apart by LPB
    const int b4 = blk & 3, h = lane % LPB;
    if (is_k) {
      if constexpr (HD == 512) {  // units of 2 bytes (t): 4 blocks x 4 units, transposed
        const uint32_t got = __shfl_xor_sync(kAll, b4 < 2 ? code[1] : code[0], 2);
        const uint32_t a0 = b4 < 2 ? code[0] : got, a1 = b4 < 2 ? got : code[1];  // units 0-1 or 2-3 of blocks b4 & 1, + 2
        const uint32_t swap = __shfl_xor_sync(kAll, __byte_perm(a0, a1, b4 & 1 ? 0x5410 : 0x7632), 1);
        const uint32_t mine = __byte_perm(a0, a1, b4 & 1 ? 0x7632 : 0x5410);
        const uint2 out = b4 & 1 ? make_uint2(__byte_perm(swap, mine, 0x5410), __byte_perm(swap, mine, 0x7632))
                                 : make_uint2(__byte_perm(mine, swap, 0x5410), __byte_perm(mine, swap, 0x7632));
        *reinterpret_cast<uint2*>(rec + kv4_k_code_at<HD>(m, p0 + 4 * b4)) = out;  // unit t = b4 of blocks 0 .. 3
      } else {  // the lane has units 2h, 2h + 1: pairs of blocks change one
        const uint32_t got = __shfl_xor_sync(kAll, code[0], LPB);
        const uint32_t out = b4 & 1 ? __byte_perm(got, code[0], 0x7632) : __byte_perm(code[0], got, 0x5410);
        *reinterpret_cast<uint32_t*>(rec + kv4_k_code_at<HD>(m, p0 + (b4 & 2) * 16 + 4 * (2 * h + (b4 & 1)))) = out;
      }
    } else {
      // 4 blocks x 4 bytes (of g), transposed: byte b4 of blocks 0 .. 3
#pragma unroll
      for (int i = 0; i < (HD == 512 ? 2 : 1); ++i) {
        uint32_t c = code[i];
        uint32_t got = __shfl_xor_sync(kAll, c, 2 * LPB);
        c = b4 & 2 ? __byte_perm(got, c, 0x7632) : __byte_perm(c, got, 0x5410);  // bytes 0-1 or 2-3 of b4 & 1, + 2
        got = __shfl_xor_sync(kAll, c, LPB);
        c = b4 & 1 ? __byte_perm(got, c, 0x7351) : __byte_perm(c, got, 0x6240);
        const int g = HD == 512 ? 4 * i + b4 : 4 * h + b4;
        *reinterpret_cast<uint32_t*>(rec + kv4_v_code_at<HD>(m, p0 + 2 * g)) = c;
      }
    }
  } else if constexpr (HD == 128) {
    if (is_k) {
      *reinterpret_cast<uint16_t*>(rec + kv4_k_code_at<HD>(m, d0)) = static_cast<uint16_t>(code[0]);
    } else {
      rec[kv4_v_code_at<HD>(m, d0)] = static_cast<uint8_t>(code[0]);
      rec[kv4_v_code_at<HD>(m, d0 + 2)] = static_cast<uint8_t>(code[0] >> 8);
    }
  } else {
    rec[is_k ? kv4_k_code_at<HD>(m, d0) : kv4_v_code_at<HD>(m, d0)] = static_cast<uint8_t>(code[0]);
  }
}

template <bool KV4>
using ArgsOf = std::conditional_t<KV4, Kv4AppendArgs, AppendArgs>;

template <typename T, int HD, bool KV4, bool IN_PLACE>
__global__ void __launch_bounds__(128, HD < 512 ? 8 : IN_PLACE ? 4 : 5) append_normrope_kernel(const __grid_constant__ ArgsOf<KV4> a) {
  constexpr int HALF = HD / 2;
  constexpr int E = HD / 64;
  constexpr bool kBF16 = sizeof(T) == 2;
  static_assert(!IN_PLACE || (kBF16 && !KV4), "the others look at no element again after its store");
  constexpr float kErrY = normrope_err_y<2 * E>();
  constexpr float kErrAB = normrope_err_pair(kDFTrigErrUnits);
  constexpr float kErrO = normrope_err_out<2 * E>();
  constexpr float kErrR = normrope_err_r<2 * E>();
  constexpr int kTabs = KV4 ? kAppendMaxTokens : 1;  // tables held at once
  __shared__ DF s_cos_all[kTabs * HALF];
  __shared__ DF s_sin_all[kTabs * HALF];
  [[maybe_unused]] int tok_pos[kAppendMaxTokens], tok_tab[kAppendMaxTokens];  // KV4: position and table of each token
  int tab = 0;  // where the current token's table begins
  auto cos_of = [&](int j) -> DF { return s_cos_all[(KV4 ? tab : 0) + j]; };
  auto sin_of = [&](int j) -> DF { return s_sin_all[(KV4 ? tab : 0) + j]; };
  __shared__ __align__(16) T s_row[KV4 ? 4 * kv4_row_at(HD) : 1];  // KV4: a finished row per warp
  __shared__ __align__(16) T s_raw[IN_PLACE ? 4 * HD : 1];  // IN_PLACE: open lanes' elements of a row per warp

  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x % a.T;
  const int b0 = (blockIdx.x / a.T) * a.tok_per_cta;
  const int b1 = min(a.B, b0 + a.tok_per_cta);
  const bool owns = a.k_in != nullptr;
  const int nrows = a.H + (owns ? 2 * a.Hkv : 0);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int row0 = blockIdx.y * a.rows_per_cta;
  const int row1 = min(nrows, row0 + a.rows_per_cta);
  const int nr = row1 - row0;
  if (nr <= 0) return;

  // Error-bound multipliers of this lane's outputs on a roped row (bound =
  // kA |y_self| + kB |y_other| + kO |o|): the rotation bound where the lane's
  // pairs rotate, the plain one where none does.  A lane straddling n_rot
  // takes the rotation bound for all its pairs, which also covers the plain ones.
  const bool lane_plain = lane * E >= a.n_rot;
  const float kA = lane_plain ? kErrY : kErrAB;
  const float kB = lane_plain ? 0.0f : kErrAB;
  const float kO = lane_plain ? 0.0f : kErrO;
  const bool all_rot = __all_sync(0xffffffffu, (lane + 1) * E <= a.n_rot);

  // This lane's cos / sin (float parts; 1 / 0 past n_rot), built per position.
  float cr[E], sr[E];
  auto build_table = [&](int pos) {
    for (int j = threadIdx.x; j < HALF; j += blockDim.x) {
      DF c = {1.0f, 0.0f}, s = {0.0f, 0.0f};
      if (j < a.n_rot) sincos_df(pos, a.inv_freq[j], c, s);
      s_cos_all[j] = c;
      s_sin_all[j] = s;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < E; ++i) {
      cr[i] = s_cos_all[lane * E + i].h;
      sr[i] = s_sin_all[lane * E + i].h;
    }
  };
  // KV4: token b's table becomes the current one.
  auto use_table = [&](int b) {
    tab = 0;
#pragma unroll
    for (int i = 1; i < kAppendMaxTokens; ++i)
      if (i == b - b0) tab = tok_tab[i] * HALF;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      cr[i] = cos_of(lane * E + i).h;
      sr[i] = sin_of(lane * E + i).h;
    }
  };

  // Where head row `row` of token (b, t) at position pos comes from and goes to.
  struct RowRef {
    const T* src;
    T* dst;
    const float* w;
    bool rope;
    bool valid;
    uint8_t* rec;  // KV4: the record of a k or v row (null: a q row, whose place is dst) and its position there
    int m;
  };
  // Where element d of a row goes: its place, or (KV4) the warp's row in shared memory.
  T* const row_buf = s_row + (KV4 ? warp * kv4_row_at(HD) : 0);
  auto at = [&](const RowRef& rr, int d) -> T* {
    if constexpr (KV4)
      return row_buf + kv4_row_at(d);
    else
      return rr.dst + d;
  };
  // (KV4: pos is the token's slot)
  auto row_ref = [&](int b, int row, int pos) -> RowRef {
    const int tok = b * a.T + t;
    RowRef rr;
    rr.rec = nullptr;
    rr.m = 0;
    if (row < a.H) {  // q head
      const size_t off = (static_cast<size_t>(tok) * a.H + row) * HD;
      rr.src = static_cast<const T*>(a.q_in) + off;
      rr.dst = static_cast<T*>(a.q_out) + off;
      rr.w = a.q_w;
      rr.rope = true;
      rr.valid = true;
    } else {
      const bool is_k = row < a.H + a.Hkv;
      const int kvh = is_k ? row - a.H : row - a.H - a.Hkv;
      rr.src = static_cast<const T*>(is_k ? a.k_in : a.v_in) + (static_cast<size_t>(tok) * a.Hkv + kvh) * HD;
      if constexpr (KV4) {
        const int slot = pos;
        rr.valid = slot >= 0 && slot < a.n_slots;
        const int in_block = slot & ((1 << a.block_shift) - 1);
        rr.dst = nullptr;
        rr.rec = static_cast<uint8_t*>(a.cache_k) +
                 kv4_record<HD>(rr.valid ? slot >> a.block_shift : 0, kvh, in_block >> 4, a.Hkv, a.block_shift);
        rr.m = in_block & 15;
      } else {
        // k / v need a cache row: the position itself, or on a sliding-window
        // ring the position modulo its capacity.
        rr.valid = pos >= 0 && (a.ring || pos < a.max_len);
        const int crow = !rr.valid ? 0 : (a.ring ? pos % a.max_len : pos);
        rr.dst = static_cast<T*>(is_k ? a.cache_k : a.cache_v) +
                 ((static_cast<size_t>(b) * a.Hkv + kvh) * a.max_len + crow) * HD;
      }
      rr.w = is_k ? a.k_w : nullptr;
      rr.rope = is_k;
    }
    return rr;
  };
  auto load_row = [&](const RowRef& rr, HalfBits<T, E>& lo, HalfBits<T, E>& hi) {
    if (!rr.valid) return;
    load_bits<E>(rr.src + lane * E, lo);
    load_bits<E>(rr.src + HALF + lane * E, hi);
  };

  // Where the elements of a row are looked at again (those of lanes with open values).
  auto again = [&](const RowRef& rr) -> const T* {
    if constexpr (IN_PLACE)
      return s_raw + warp * HD;
    else
      return rr.src;
  };

  // Values of row rr that the float32 evaluation could not decide (bit k of
  // need: element k of the lane's 2E, lower half first), evaluated again in
  // double-float from the row's inverse rms rd and stored over the fast ones.
  // One element per pass, so the loop stays short for the usual 0-2 bits.
  auto fix_elems = [&](const RowRef& rr, uint32_t need, DF rd) {
#pragma unroll 1
    while (need != 0) {
      const int k = __ffs(need) - 1;
      need &= need - 1;
      const bool lower = k < E;
      const int j = lane * E + (lower ? k : k - E);
      const int self = lower ? j : HALF + j, other = lower ? HALF + j : j;
      const float xs = static_cast<float>(again(rr)[self]);
      float v;
      if (rr.rope) {
        const float xo = static_cast<float>(again(rr)[other]);
        const float ws = rr.w != nullptr ? rr.w[self] : 1.0f, wo = rr.w != nullptr ? rr.w[other] : 1.0f;
        v = normrope_exact_bf16_inl(xs, ws, xo, wo, rd, j < a.n_rot, lower, cos_of(j), sin_of(j));
      } else {
        v = df_round_bf16(df_mul_f(rd, xs));
      }
      *at(rr, self) = static_cast<T>(v);
    }
  };

  // Second stage for the values of row rr the float32 evaluation left open
  // (bits of need, as for fix_elems): the same float inverse rms r times the
  // row's inner products in double-float.  That value is off from the exact
  // one by r's own error (and 2^-40 of the terms), much less than the float32
  // evaluation, so it decides most of them; the bits still open are returned.
  auto refine = [&](const RowRef& rr, uint32_t need, float r) -> uint32_t {
    uint32_t open = 0;
#pragma unroll 1
    while (need != 0) {
      const int k = __ffs(need) - 1;
      need &= need - 1;
      const bool lower = k < E;
      const int j = lane * E + (lower ? k : k - E);
      const int self = lower ? j : HALF + j, other = lower ? HALF + j : j;
      const float xs = static_cast<float>(again(rr)[self]);
      DF inner = {xs, 0.0f};
      float mag = fabsf(xs);
      if (rr.rope) {
        const float ws = rr.w != nullptr ? rr.w[self] : 1.0f;
        inner = two_prod(xs, ws);
        mag = fabsf(inner.h);
        if (j < a.n_rot) {
          const float xo = static_cast<float>(again(rr)[other]);
          const float wo = rr.w != nullptr ? rr.w[other] : 1.0f;
          const DF po = two_prod(xo, wo);
          mag += fabsf(po.h);
          inner = df_add(df_mul(inner, cos_of(j)), df_mul(po, lower ? df_neg(sin_of(j)) : sin_of(j)));
        }
      }
      const DF v = df_mul_f(inner, r);
      const float e = fmaf(kErrR, fabsf(v.h), 0x1.0p-40f * r * mag);
      if (fabsf((v.h - bf16_midpoint(v.h)) + v.l) > e)
        *at(rr, self) = static_cast<T>(df_round_bf16(v));
      else
        open |= 1u << k;
    }
    return open;
  };

  // One row: float32 evaluation, stored.  For bf16, a value whose rounding
  // the float32 evaluation cannot decide (Ziv's test against its error bound)
  // is then decided in double-float (refine, then fix_elems).  all_rot (warp-uniform):
  // every lane's pairs rotate, so both outputs of a pair share one bound.
  auto do_row = [&](const RowRef& rr, const HalfBits<T, E>& lo, const HalfBits<T, E>& hi, auto all_rot_tag) {
    [[maybe_unused]] constexpr bool kAllRot = decltype(all_rot_tag)::value;
    if (!rr.valid) return;
    float x[2 * E], o[2 * E];
    unpack_bits<E>(lo, x);
    unpack_bits<E>(hi, x + E);
    const float sf = row_sumsq_f32<2 * E>(x);
    const float r = inv_rms_f32(sf, HD, a.eps);
    [[maybe_unused]] uint32_t need = 0;
    if (rr.rope) {
      float wl[E], wh[E], ya[E], yb[E];
      if (rr.w != nullptr) {
        load_elems<E>(rr.w + lane * E, wl);
        load_elems<E>(rr.w + HALF + lane * E, wh);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) wl[i] = wh[i] = 1.0f;
      }
      scale_elems<E>(ya, x, r, wl);
      scale_elems<E>(yb, x + E, r, wh);
      rotate_elems<E>(o, o + E, ya, yb, cr, sr);
      if constexpr (kBF16) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float aa = fabsf(ya[i]), ab = fabsf(yb[i]);
          float ea, eb;
          if constexpr (kAllRot) {
            const float shared = kErrAB * (aa + ab);
            ea = fmaf(kErrO, fabsf(o[i]), shared);
            eb = fmaf(kErrO, fabsf(o[E + i]), shared);
          } else {
            ea = fmaf(kO, fabsf(o[i]), fmaf(kB, ab, kA * aa));
            eb = fmaf(kO, fabsf(o[E + i]), fmaf(kB, aa, kA * ab));
          }
          need |= (bf16_decided(o[i], ea) ? 0u : 1u) << i;
          need |= (bf16_decided(o[E + i], eb) ? 0u : 1u) << (E + i);
        }
      }
    } else {  // v head: weight-less norm, no rotation
      scale_elems<E>(o, x, r, nullptr);
      scale_elems<E>(o + E, x + E, r, nullptr);
      if constexpr (kBF16) {
#pragma unroll
        for (int k = 0; k < 2 * E; ++k) need |= (bf16_decided(o[k], kErrY * fabsf(o[k])) ? 0u : 1u) << k;
      }
    }
    if constexpr (IN_PLACE) {
      if (need != 0) {
        store_bits<E>(s_raw + warp * HD + lane * E, lo);
        store_bits<E>(s_raw + warp * HD + HALF + lane * E, hi);
      }
    }
    store_elems<E>(at(rr, lane * E), o);
    store_elems<E>(at(rr, HALF + lane * E), o + E);
    if constexpr (kBF16) {
      if (__any_sync(0xffffffffu, need != 0)) {
        need = refine(rr, need, r);
        if (__any_sync(0xffffffffu, need != 0))
          fix_elems(rr, need, inv_rms_df(row_sumsq_split<2 * E, HD>(x, sf), HD, a.eps));
      }
    }
    if constexpr (KV4) {
      __syncwarp();
      if (rr.rec != nullptr) {
        kv4_store_row<HD>(row_buf, rr.rec, rr.m, rr.rope, rr.rope ? a.k_mul : 1.0f, lane);
      } else {
        constexpr int C = HD >= 256 ? 8 : HD / 32;  // elements per copy
        using V = std::conditional_t<C == 8, uint4, std::conditional_t<C == 4, uint2, uint32_t>>;
#pragma unroll
        for (int d = lane * C; d < HD; d += 32 * C)
          *reinterpret_cast<V*>(rr.dst + d) = *reinterpret_cast<const V*>(row_buf + kv4_row_at(d));
      }
      __syncwarp();
    }
  };

  // Rows of tokens [bA, bB) (all at position pos), flattened in (b, row)
  // order; warp w takes items w, w + 4, ... (KV4 with four tokens: those of
  // token w).  The next item's loads are issued before the current one is computed.
  // `then` runs after the first item's loads have been issued.
  auto run = [&](int bA, int bB, int pos, auto then) {
    int b = bA, row = row0 + warp, stride = 4;
    if (KV4 && bB - bA == 4) {  // a token per warp: its cos / sin are loaded once
      b = bA + warp;
      bB = b + 1;
      row = row0;
      stride = 1;
    }
    while (row >= row1 && b < bB) { row -= nr; ++b; }
    RowRef rr = {};
    HalfBits<T, E> lo, hi;
    [[maybe_unused]] int b_tab = -1;
    if constexpr (KV4) {
      if (b < bB && owns) pos = a.slots[b * a.T + t];
    }
    if (b < bB) {
      rr = row_ref(b, row, pos);
      load_row(rr, lo, hi);
    }
    then();
    while (b < bB) {
      int bn = b, rn = row + stride;
      while (rn >= row1 && bn < bB) { rn -= nr; ++bn; }
      RowRef rrn = {};
      HalfBits<T, E> lon, hin;
      [[maybe_unused]] int pos_n = pos;
      if (bn < bB) {
        if constexpr (KV4) {
          if (bn != b && owns) pos_n = a.slots[bn * a.T + t];
        }
        rrn = row_ref(bn, rn, pos_n);
        load_row(rrn, lon, hin);
      }
      if constexpr (KV4) {
        if (b != b_tab) use_table(b_tab = b);
        rr = row_ref(b, row, pos);  // (again, rather than kept from the load: its registers)
      }
      if (all_rot)
        do_row(rr, lo, hi, std::true_type());
      else
        do_row(rr, lo, hi, std::false_type());
      b = bn;
      row = rn;
      if constexpr (KV4)
        pos = pos_n;
      else
        rr = rrn;
      lo = lon;
      hi = hin;
    }
  };

  if constexpr (KV4) {
    // A table per distinct position (neighbours that agree share one), all of
    // them built at once while the first rows are on their way, so that rows of
    // all tokens follow each other.
#pragma unroll
    for (int i = 0; i < kAppendMaxTokens; ++i) {
      tok_pos[i] = a.positions[min(b0 + i, b1 - 1) * a.T + t];
      tok_tab[i] = i == 0 ? 0 : tok_tab[i - 1] + (tok_pos[i] != tok_pos[i - 1]);
    }
    run(b0, b1, 0, [&] {
      const int ntab = tok_tab[kAppendMaxTokens - 1] + 1;
      for (int idx = threadIdx.x; idx < ntab * HD; idx += blockDim.x) {
        const int j = (idx >> 1) % HALF, part = idx & 1, tb = idx / HD, at = tb * HALF + j;
        int pos = tok_pos[0];
#pragma unroll
        for (int i = 1; i < kAppendMaxTokens; ++i)
          if (tok_tab[i] == tb) pos = tok_pos[i];
        if (j < a.n_rot) {
          bool to_cos;
          const DF v = sincos_df_part(pos, a.inv_freq[j], part, to_cos);
          (to_cos ? s_cos_all : s_sin_all)[at] = v;
        } else if (part == 0) {
          s_cos_all[at] = DF{1.0f, 0.0f};
        } else {
          s_sin_all[at] = DF{0.0f, 0.0f};
        }
      }
      __syncthreads();
    });
    return;
  }
  // One cos/sin table serves every token of the CTA when their positions
  // agree (the usual prefill case); otherwise tokens go one at a time.
  const int p0 = a.positions[b0 * a.T + t];
  bool same = true;
  for (int b = b0 + 1; b < b1; ++b) same = same && a.positions[b * a.T + t] == p0;
  if (same) {
    build_table(p0);
    run(b0, b1, p0, [] {});
  } else {
    for (int b = b0; b < b1; ++b) {
      if (b > b0) __syncthreads();  // every warp is done with the previous table
      const int pos = a.positions[b * a.T + t];
      build_table(pos);
      run(b, b + 1, pos, [] {});
    }
  }
}

template <typename Kern, typename Args>
cudaError_t launch_pdl(Kern kern, dim3 grid, cudaStream_t s, const Args& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename T, bool KV4, bool IN_PLACE>
cudaError_t launch_t(const ArgsOf<KV4>& a, cudaStream_t s) {
  const int nrows = a.H + (a.k_in ? 2 * a.Hkv : 0);
  dim3 grid(a.T * ((a.B + a.tok_per_cta - 1) / a.tok_per_cta), (nrows + a.rows_per_cta - 1) / a.rows_per_cta);
  switch (a.hd) {
    case 64: return launch_pdl(append_normrope_kernel<T, 64, KV4, IN_PLACE>, grid, s, a);
    case 128: return launch_pdl(append_normrope_kernel<T, 128, KV4, IN_PLACE>, grid, s, a);
    case 256: return launch_pdl(append_normrope_kernel<T, 256, KV4, IN_PLACE>, grid, s, a);
    case 512: return launch_pdl(append_normrope_kernel<T, 512, KV4, IN_PLACE>, grid, s, a);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int dtype, cudaStream_t s) {
  if (dtype != 1) return launch_t<float, false, false>(a, s);
  return a.q_in == a.q_out ? launch_t<__nv_bfloat16, false, true>(a, s) : launch_t<__nv_bfloat16, false, false>(a, s);
}

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t s) {
  return launch_t<__nv_bfloat16, true, false>(a, s);
}

}  // namespace g4
