// The append with positions of several axes (g4_kv_append_normrope_axes): per-head
// RMSNorm, rotate_half RoPE whose pair j turns by the position of its axis, k and v
// written to the cache's rows.  What is stored is what g4_append.cu stores, in bf16
// the correctly rounded real result, but it is found with fewer instructions:
//
//   * cos and sin come from float32 polynomials on an angle reduced in two floats, off by
//     at most 1.23 x 2^-24 for angles below 2^20 (a brute-force comparison with extended
//     precision; a double-float table costs six times as much, and a token whose axes
//     differ shares its table with no other).  Only a value that they leave open
//     meets cos and sin in double-float.
//   * A lane owns chunks of up to 4 neighbouring pairs, 128 pairs apart, so that the pairs that a
//     partial rotary leaves as they are lie in chunks of their own, which skip
//     the rotation and its wider test.  (In float32, where nothing is tested, pairs
//     and tables are g4_append.cu's, and so are the results, bit for bit.)
//   * Ziv's test on an unrotated value, whose error is a few units in its own last
//     place, is made on the integers' low halves, two values at a time: a low half
//     lies near a rounding boundary or it does not.  A rotated one is compared
//     with one bound per pair.
//   * A warp takes tokens by itself, table and all: no barrier of the CTA is left.  Their rows come
//     by bulk copies ahead of their use, positions and cache rows a token ahead.
//
// A value left open (a third of the rows have one) is formed again in double-float, from the
// row's inverse rms and its elements' exact products, and stored over the first one.
// q_out may be q_in: what is read again after a store is the row's copy in shared memory.
//
// Measured (device time): 8 x 2048 tokens of 8 + 2 + 2 rows of 512, an eighth of each
// rotated, 125 us, 2.9 TB/s (369 MB; 145 us with g4_append.cu's arithmetic and a
// table for each token); of 256, all rotated, 105 us; float32 with as many bytes 75 us,
// 4.9 TB/s; the new tokens of 64 sequences, head_dim 256, 4.9 us (6.2).  Bound by
// instruction issue: some 320 per row, and 100 for values left open; small launches by the
// chain of loads.
#include "g4_device.cuh"
#include "g4_internal.h"
#include "g4_normrope.cuh"

namespace g4 {
namespace {

constexpr int kWarps = 4;
constexpr float kTrigUnits = 1.5f;  // bound on the error of sincos_f32 in units of 2^-24

// sincos_df as a call of its own, {cos, sin}: rarely needed, and long.
static __device__ __noinline__ float4 sincos_exact(int p, float f) {
  DF c, s;
  sincos_df(p, f, c, s);
  return make_float4(c.h, c.l, s.h, s.l);
}

// cos and sin of p * f: the exact product less the nearest multiple k of pi/2 (three floats), Taylor polynomials.
__device__ __forceinline__ bool angle_is_near(int p, float f) {
  return fabsf(static_cast<float>(p) * f) < 0x1.0p20f && p < (1 << 24) && p > -(1 << 24);
}
__device__ __forceinline__ float2 sincos_f32(int p, float f) {
  const float pf = static_cast<float>(p);
  const float th = pf * f, tl = fmaf(pf, f, -th);
  // (k no longer the nearest, or p not exact)
  if (!angle_is_near(p, f)) {
    const float4 v = sincos_exact(p, f);
    return make_float2(v.x, v.z);
  }
  const float k = rintf(th * 0x1.45f306p-1f);  // 2 / pi
  constexpr float P1 = 0x1.921fb6p+0f, P2 = -0x1.777a5cp-25f, P3 = -0x1.ee59dap-50f;  // pi / 2
  const float ah = k * P1, al = fmaf(k, P1, -ah);
  const float r = (th - ah) + fmaf(-k, P3, fmaf(-k, P2, tl - al));
  const float z = r * r;
  float sn = fmaf(z, 0x1.71de3ap-19f, -0x1.a01a02p-13f);
  sn = fmaf(z, sn, 0x1.111112p-7f);
  sn = fmaf(z, sn, -0x1.555556p-3f);
  sn = fmaf(r * z, sn, r);
  float cs = fmaf(z, -0x1.27e4fcp-22f, 0x1.a01a02p-16f);
  cs = fmaf(z, cs, -0x1.6c16c2p-10f);
  cs = fmaf(z, cs, 0x1.555556p-5f);
  cs = fmaf(z, cs, -0.5f);
  cs = fmaf(z, cs, 1.0f);
  const int q = static_cast<int>(k) & 3;
  const float c = q & 1 ? sn : cs, s = q & 1 ? cs : sn;
  return make_float2(q == 1 || q == 2 ? -c : c, q >= 2 ? -s : s);
}

// The same with two floats each, off by at most 0.32 x 2^-24: the reduced angle in double-float, the heads of both
// series exact, their tails in float32.  A third of sincos_df's instructions.
constexpr float kMidErr = 0x1.0p-24f;  // (three times that)
__device__ __forceinline__ void sincos_mid(int p, float f, DF& c, DF& s) {
  int q;
  const DF r = reduce_angle_df(p, f, q);
  const float z = r.h * r.h, zl = fmaf(2.0f * r.h, r.l, fmaf(r.h, r.h, -z));
  float ps = fmaf(z, 0x1.71de3ap-19f, -0x1.a01a02p-13f);
  ps = fmaf(z, ps, 0x1.111112p-7f);
  ps = fmaf(z, ps, -0x1.555556p-3f);
  const DF sn = fast_two_sum(r.h, fmaf(r.h * z, ps, r.l * fmaf(z, -0.5f, 1.0f)));
  float pc = fmaf(z, -0x1.27e4fcp-22f, 0x1.a01a02p-16f);
  pc = fmaf(z, pc, -0x1.6c16c2p-10f);
  pc = fmaf(z, pc, 0x1.555556p-5f);
  DF cs = fast_two_sum(1.0f, -0.5f * z);
  cs = fast_two_sum(cs.h, cs.l + fmaf(z * z, pc, -0.5f * zl));
  c = q & 1 ? sn : cs;
  s = q & 1 ? cs : sn;
  if (q == 1 || q == 2) c = df_neg(c);
  if (q >= 2) s = df_neg(s);
}

template <typename T, int HD>
struct AxCfg {
  static constexpr int HALF = HD / 2;
  static constexpr int E = HD / 64;              // pairs per lane
  static constexpr int CW = sizeof(T) == 2 && E > 4 ? 4 : E;  // neighbouring ones
  static constexpr int NCH = E / CW;             // chunks
  static constexpr int SPAN = 32 * CW;           // pairs of the warp per chunk
  static constexpr int ROW_B = HD * static_cast<int>(sizeof(T));
  // Where a warp has several units, rows come by bulk copies through a ring of its own.
  static constexpr int RPC = (HD >= 512 ? 4096 : 2048) / ROW_B;  // rows per copy, at most
  static constexpr int NST = HD >= 512 ? 2 : 3;
  static constexpr int RING_B = NST * RPC * ROW_B;
  // CTAs per SM.  (With 8 of 64 registers each two launches of a few rows fit side by side: 3 x 101 float32 tokens of
  // head_dim 128 3.2 us against 4.6 with 6.  512: 5 of them spill, 140 us against 123 at 8 x 2048 tokens.)
  static constexpr int RESIDENT = HD >= 512 ? 4 : HD >= 256 ? 6 : 8;
};

// y[i] = x[i] f (or x[i] f[i]), two at a time.
template <int N>
__device__ __forceinline__ void times(float* x, float f) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 v = __fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(f, f));
      x[i] = v.x;
      x[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] *= f;
  }
}
template <int N>
__device__ __forceinline__ void times(float* x, const float* f) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 v = __fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(f[i], f[i + 1]));
      x[i] = v.x;
      x[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] *= f[i];
  }
}

template <typename T, int HD>
__global__ void __launch_bounds__(kWarps * 32, AxCfg<T, HD>::RESIDENT) append_axes_kernel(const __grid_constant__ AxesAppendArgs a) {
  using C = AxCfg<T, HD>;
  constexpr int HALF = C::HALF, E = C::E, CW = C::CW, NCH = C::NCH;
  constexpr bool kBF16 = sizeof(T) == 2;
  constexpr float kErrY = normrope_err_y<2 * E>();
  constexpr float kErrAB = normrope_err_pair(kTrigUnits);
  constexpr float kErrO = normrope_err_out<2 * E>();
  // An unrotated value's error in units of its last place: the integer test's window, which takes in one more for the
  // carry between two halves.
  constexpr int kUlps = static_cast<int>(kErrY * 0x1.0p24f) + 1;
  constexpr uint32_t kBoth = 0x00010001u;
  static_assert(E <= 8, "two squares per sum at most");
  extern __shared__ __align__(128) uint8_t s_ring[];  // [warp][NST][RPC] rows
  __shared__ float s_freq[HALF];
  __shared__ uint8_t s_axis[HALF];
  __shared__ __align__(16) float s_cs_all[kWarps][3 * HALF];  // a token's table: cos, sin and -sin of each pair
  __shared__ uint64_t s_bar[kWarps][C::NST];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_rot = a.n_rot, n_tab = min(HALF, (n_rot + C::SPAN - 1) / C::SPAN * C::SPAN);  // whole chunks
  // (read once per CTA: lanes that read elements of their own from the arguments take turns)
  for (int j = threadIdx.x; j < n_tab; j += kWarps * 32) {
    s_freq[j] = j < n_rot ? a.inv_freq[j] : 0.0f;
    s_axis[j] = j < n_rot ? a.axis[j] : 0;
  }
  uint64_t* bars = s_bar[warp];
  if (lane == 0) {
    for (int i = 0; i < C::NST; ++i) mbar_init(smem_u32(&bars[i]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  uint8_t* ring = s_ring + warp * C::RING_B;
  float* cs = s_cs_all[warp];
  const bool owns = a.k_in != nullptr;
  const int nq = a.H, nk = a.H + a.Hkv;  // rows of a token: q below nq, k below nk, then v
  const int nrows = owns ? nk + a.Hkv : nq;
  const int parts = (nrows + a.rows_per_unit - 1) / a.rows_per_unit;  // units of a token
  const int tokens = a.B * a.T;
  const long long units = static_cast<long long>(tokens) * parts;
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  const long long unit0 = static_cast<long long>(blockIdx.x) * kWarps + warp;
  auto token_of = [&](long long unit) {
    if (parts == 1) return static_cast<int>(unit);
    if (units <= 0x7fffffff) return static_cast<int>(unit) / parts;  // (a division in 64 bits takes several times as long)
    return static_cast<int>(unit / parts);
  };
  auto first_row = [&](long long unit, int tok) {
    return parts == 1 ? 0 : static_cast<int>(unit - static_cast<long long>(tok) * parts) * a.rows_per_unit;
  };
  // rows of one copy: neighbours of one tensor
  auto run_of = [&](int row, int end) { return min(C::RPC, min(end, row < nq ? nq : row < nk ? nk : nrows) - row); };
  auto pair_at = [&](int c) { return c * C::SPAN + lane * CW; };  // the lane's first pair of a chunk

  auto source = [&](int tok, int row) -> const T* {
    if (row < nq) return static_cast<const T*>(a.q_in) + (static_cast<size_t>(tok) * nq + row) * HD;
    return static_cast<const T*>(row < nk ? a.k_in : a.v_in) + (static_cast<size_t>(tok) * a.Hkv + row - (row < nk ? nq : nk)) * HD;
  };

  // The copies of this warp's rows, unit by unit, ahead of their use (lane 0's).
  long long ask_unit = unit0;
  int ask_tok = 0, ask_row = 0, ask_end = 0, ask_slot = 0;
  auto ask = [&]() {
    if (ask_row == ask_end) {
      if (ask_unit >= units) return;
      ask_tok = token_of(ask_unit);
      ask_row = first_row(ask_unit, ask_tok);
      ask_end = min(nrows, ask_row + a.rows_per_unit);
      ask_unit += step;
    }
    const int n = run_of(ask_row, ask_end);
    const uint32_t bar = smem_u32(&bars[ask_slot]), bytes = static_cast<uint32_t>(n) * C::ROW_B;
    mbar_arrive_expect_tx(bar, bytes);
    bulk_g2s(smem_u32(ring + ask_slot * C::RPC * C::ROW_B), source(ask_tok, ask_row), bytes, bar);
    ask_row += n;
    if (++ask_slot == C::NST) ask_slot = 0;
  };
  // What a unit is placed by.
  struct Place {
    int pos[4], row;
  };
  auto place_of = [&](long long unit) {
    Place p;
    const int tok = token_of(unit);
#pragma unroll
    for (int x = 0; x < 4; ++x) p.pos[x] = x < a.n_axes ? a.positions[static_cast<size_t>(x) * tokens + tok] : 0;
    p.row = owns ? a.rows[tok] : -1;
    return p;
  };
  if (unit0 >= units) return;
  // A single unit's rows are read where they are: a copy would only be waited for.  Not in place, though: values left
  // open are formed from the inputs again after the others have been stored.
  const bool staged = units > step || a.q_in == a.q_out;
  if (staged) {
    if (lane == 0)
      for (int i = 0; i < C::NST; ++i) ask();
  }
  // The unit's first row, where it is not copied ahead: on its way in registers while the table is made.
  float lo_1[E], hi_1[E];
  if (!staged) {
    const int tok = token_of(unit0);
    const T* first = source(tok, first_row(unit0, tok));
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      load_elems<CW>(first + pair_at(c), lo_1 + c * CW);
      load_elems<CW>(first + HALF + pair_at(c), hi_1 + c * CW);
    }
  }
  Place now = place_of(unit0);
  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;

  for (long long unit = unit0; unit < units && ok; unit += step) {
    const int tok = token_of(unit), row0 = first_row(unit, tok);
    const int row1 = min(nrows, row0 + a.rows_per_unit);
    Place then = {};
    if (unit + step < units) then = place_of(unit + step);  // (on its way while this unit is worked on)
    auto position = [&](int x) { return x == 0 ? now.pos[0] : x == 1 ? now.pos[1] : x == 2 ? now.pos[2] : now.pos[3]; };
    __syncwarp();  // (the last unit's table has been read)
    if (row0 < nk) {
      for (int j = lane; j < n_tab; j += 32) {
        float2 v = make_float2(1.0f, 0.0f);
        if (j < n_rot) {
          const int p = position(s_axis[j]);
          if constexpr (kBF16) {
            v = sincos_f32(p, s_freq[j]);
          } else {
            DF c, s;
            sincos_df(p, s_freq[j], c, s);
            v = make_float2(c.h, s.h);
          }
        }
        cs[j] = v.x;
        cs[HALF + j] = v.y;
        cs[2 * HALF + j] = -v.y;
      }
      __syncwarp();
    }
    const bool kept = now.row >= 0 && (a.ring || now.row < a.max_len);
    const size_t place = (static_cast<size_t>(tok / a.T) * a.Hkv * a.max_len + (!kept ? 0 : a.ring ? now.row % a.max_len : now.row)) * HD;

    float w_lo[E], w_hi[E];
    int w_of = -1;  // whose weights they are: 0 q's, 1 k's, 2 v's (ones)
    for (int row = row0; row < row1;) {
      const int n = run_of(row, row1);
      if (staged && !warp_wait(smem_u32(&bars[slot]), phase, a.err)) {
        ok = false;
        break;
      }
      const int kind = row < nq ? 0 : row < nk ? 1 : 2;
      const T* in = staged ? reinterpret_cast<const T*>(ring + slot * C::RPC * C::ROW_B) : source(tok, row);
      const float* w = kind == 0 ? a.q_w : a.k_w;
      if (kind != w_of && (kind == 0 || kept)) {
        w_of = kind;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          if (kind < 2) {
            load_elems<CW>(w + pair_at(c), w_lo + c * CW);
            load_elems<CW>(w + HALF + pair_at(c), w_hi + c * CW);
          } else {
#pragma unroll
            for (int i = 0; i < CW; ++i) w_lo[c * CW + i] = w_hi[c * CW + i] = 1.0f;
          }
        }
      }
      T* dst = static_cast<T*>(a.q_out) + (static_cast<size_t>(tok) * nq + row) * HD;
      size_t stride = HD;
      if (kind > 0) {
        stride = static_cast<size_t>(a.max_len) * HD;
        dst = static_cast<T*>(kind == 1 ? a.cache_k : a.cache_v) + place + (row - (kind == 1 ? nq : nk)) * stride;
      }
      const bool rope = kind < 2;
      const int todo_rows = kind == 0 || kept ? n : 0;
#pragma unroll 1
      for (int i_row = 0; i_row < todo_rows; ++i_row, in += HD, dst += stride) {
        float lo[E], hi[E];
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          if (!staged && row == row0 && i_row == 0) {
#pragma unroll
            for (int i = c * CW; i < (c + 1) * CW; ++i) {
              lo[i] = lo_1[i];
              hi[i] = hi_1[i];
            }
          } else {
            load_elems<CW>(in + pair_at(c), lo + c * CW);
            load_elems<CW>(in + HALF + pair_at(c), hi + c * CW);
          }
        }
        float sf;
        if constexpr (kBF16 && E >= 2) {
          // The sum of squares: squares of bf16 are exact in float32, so 2 E of them take log2(2 E) roundings, as
          // row_sumsq_f32's: two neighbours side by side, 4 sums of them, the second of each added by an fma.
          constexpr int NA = E < 4 ? E : 4;
          float2 acc[NA];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float* x = e % 2 ? hi + e - 1 : lo + e;
            const float2 v = make_float2(x[0], x[1]);
            acc[e % NA] = e < NA ? __fmul2_rn(v, v) : __ffma2_rn(v, v, acc[e % NA]);
          }
#pragma unroll
          for (int h = NA / 2; h >= 1; h /= 2)
#pragma unroll
            for (int i = 0; i < h; ++i) acc[i] = __fadd2_rn(acc[i], acc[i + h]);
          sf = acc[0].x + acc[0].y;
#pragma unroll
          for (int x = 16; x >= 1; x >>= 1) sf += __shfl_xor_sync(0xffffffffu, sf, x);
        } else {
          float x[2 * E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            x[e] = lo[e];
            x[E + e] = hi[e];
          }
          sf = row_sumsq_f32<2 * E>(x);
        }
        const float r = inv_rms_f32(sf, HD, a.eps);

        float oa[E], ob[E];
        uint32_t need = 0;  // pair e's values whose rounding may not be decided: bits e (lower) and 16 + e
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          float ya[CW], yb[CW];
#pragma unroll
          for (int i = 0; i < CW; ++i) {
            ya[i] = lo[c * CW + i];
            yb[i] = hi[c * CW + i];
          }
          times<CW>(ya, r);
          times<CW>(yb, r);
          times<CW>(ya, w_lo + c * CW);  // (v's weights are ones, which change nothing)
          times<CW>(yb, w_hi + c * CW);
          if (rope && c * C::SPAN < n_tab) {
            float cj[CW], sj[CW], nj[CW], ta[CW], tb[CW];
            load_elems<CW>(cs + pair_at(c), cj);
            load_elems<CW>(cs + HALF + pair_at(c), sj);
            load_elems<CW>(cs + 2 * HALF + pair_at(c), nj);
#pragma unroll
            for (int i = 0; i < CW; ++i) {
              ta[i] = yb[i];
              tb[i] = ya[i];
            }
            times<CW>(ta, nj);
            times<CW>(tb, sj);
            if constexpr (CW % 2 == 0) {
#pragma unroll
              for (int i = 0; i < CW; i += 2) {
                const float2 cc = make_float2(cj[i], cj[i + 1]);
                const float2 va = __ffma2_rn(make_float2(ya[i], ya[i + 1]), cc, make_float2(ta[i], ta[i + 1]));
                const float2 vb = __ffma2_rn(make_float2(yb[i], yb[i + 1]), cc, make_float2(tb[i], tb[i + 1]));
                oa[c * CW + i] = va.x;
                oa[c * CW + i + 1] = va.y;
                ob[c * CW + i] = vb.x;
                ob[c * CW + i + 1] = vb.y;
              }
            } else {
              oa[c] = fmaf(ya[0], cj[0], ta[0]);
              ob[c] = fmaf(yb[0], cj[0], tb[0]);
            }
            if constexpr (kBF16) {
#pragma unroll
              for (int i = 0; i < CW; ++i) {
                const int e = c * CW + i;
                const float err = (kErrAB + kErrO) * (fabsf(ya[i]) + fabsf(yb[i]));  // (|o| is at most that sum)
                if (!(fabsf(oa[e] - bf16_midpoint(oa[e])) > err)) need |= 1u << e;
                if (!(fabsf(ob[e] - bf16_midpoint(ob[e])) > err)) need |= 0x10000u << e;
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < CW; ++i) {
              const int e = c * CW + i;
              oa[e] = ya[i];
              ob[e] = yb[i];
              if constexpr (kBF16) {
                // low halves less 2^15, plus kUlps: 0 .. 2 kUlps (+ 1) near a boundary
                const uint32_t t = __byte_perm(__float_as_uint(ya[i]), __float_as_uint(yb[i]), 0x5410) + (0x8000u + kUlps) * kBoth;
                need |= (~((t | 0x80008000u) - (2 * kUlps + 2) * kBoth) & ~t & 0x80008000u) >> (15 - e);
              }
            }
          }
        }

#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          store_elems<CW>(dst + pair_at(c), oa + c * CW);
          store_elems<CW>(dst + HALF + pair_at(c), ob + c * CW);
        }

        if constexpr (kBF16) {
          if (__any_sync(0xffffffffu, need != 0)) {
            // Those again, from the row's inverse rms and its elements' exact products in double-float.
            DF rd;
            {
              float x[2 * E];
#pragma unroll
              for (int e = 0; e < E; ++e) {
                x[e] = lo[e];
                x[E + e] = hi[e];
              }
              rd = inv_rms_df(row_sumsq_split<2 * E, HD>(x, sf), HD, a.eps);
            }
#pragma unroll 1
            for (; need != 0; need &= need - 1) {
              const int k = __ffs(need) - 1, e = k & 15;
              const bool lower = k < 16;
              const int j = e / CW * C::SPAN + lane * CW + e % CW;
              const int self = lower ? j : HALF + j, other = lower ? HALF + j : j;
              const DF own = two_prod(static_cast<float>(in[self]), rope ? w[self] : 1.0f);
              DF v = df_mul(own, rd);
              if (rope && j < n_rot) {
                const DF po = two_prod(static_cast<float>(in[other]), w[other]);
                auto turned = [&](DF cj, DF sj) {
                  return df_mul(df_add(df_mul(own, cj), df_mul(po, lower ? df_neg(sj) : sj)), rd);
                };
                const int at = position(s_axis[j]);
                const float f = s_freq[j];
                bool decided = angle_is_near(at, f);
                if (decided) {
                  DF cj, sj;
                  sincos_mid(at, f, cj, sj);
                  v = turned(cj, sj);
                  decided = fabsf((v.h - bf16_midpoint(v.h)) + v.l) > kMidErr * rd.h * (fabsf(own.h) + fabsf(po.h));
                }
                if (!decided) {
                  const float4 t = sincos_exact(at, f);
                  v = turned(DF{t.x, t.y}, DF{t.z, t.w});
                }
              }
              dst[self] = static_cast<T>(df_round_bf16(v));
            }
          }
        }
      }
      row += n;
      if (staged) {
        if (++slot == C::NST) {
          slot = 0;
          phase ^= 1u;
        }
        __syncwarp();  // (every lane is done with the copy's rows)
        if (lane == 0) ask();
      }
    }
    now = then;
  }
  // After a wait that gave up: wait (with a limit) for the copies still in flight.
  if (!ok)
    for (int i = 0; i < C::NST; ++i) {
      warp_wait(smem_u32(&bars[slot]), phase, nullptr);
      if (++slot == C::NST) {
        slot = 0;
        phase ^= 1u;
      }
    }
}

template <typename T, int HD>
cudaError_t launch_hd(const AxesAppendArgs& a, cudaStream_t s) {
  constexpr int smem = kWarps * AxCfg<T, HD>::RING_B;
  const cudaError_t e = set_smem_limit_once<append_axes_kernel<T, HD>>(smem);
  if (e != cudaSuccess) return e;
  const int nrows = a.H + (a.k_in != nullptr ? 2 * a.Hkv : 0);
  const long long units = static_cast<long long>(a.B) * a.T * ((nrows + a.rows_per_unit - 1) / a.rows_per_unit);
  const long long ctas = (units + kWarps - 1) / kWarps, resident = static_cast<long long>(sm_count()) * AxCfg<T, HD>::RESIDENT;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas < resident ? ctas : resident));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_axes_kernel<T, HD>, a);
}

template <typename T>
cudaError_t launch_t(const AxesAppendArgs& a, cudaStream_t s) {
  switch (a.hd) {
    case 64: return launch_hd<T, 64>(a, s);
    case 128: return launch_hd<T, 128>(a, s);
    case 256: return launch_hd<T, 256>(a, s);
    case 512: return launch_hd<T, 512>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_append_axes(const AxesAppendArgs& a, int dtype, cudaStream_t s) {
  return dtype == 1 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
}

}  // namespace g4
