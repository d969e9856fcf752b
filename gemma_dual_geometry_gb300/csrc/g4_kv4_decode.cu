// Decode attention over the paged 4-bit KV cache: one query per sequence,
// split over the key range (split-KV), HBM-bound.
//
// out_h = sum_j p_j v_j / sum_j p_j,  p_j = 2^(c (q_h . k_j) - m),  over the keys
// [max(0, L - window), L) (all L on full layers), c = attn_scale log2(e).
//
// One CTA per (split, kv head, sequence), all G <= 8 query heads of the kv
// head together, so a record of the cache is read once.  A record (16
// positions, 18 head_dim bytes) is one bulk copy; every warp owns a ring of
// stages and takes its CTA's records in turn.  At 4.5 bits per element an SM's
// share of HBM is ~42 elements per clock, each of which meets 8 (padded)
// heads twice: more multiply-adds than the CUDA cores have, so both products
// run on mma.sync m16n8k16 (fp16 operands, float32 sums), whose 16 x 16 operand
// is a record's scale block and whose 8 columns are the heads:
//   S^T[16 positions][8 heads] += s . (K[16 x 16] Q^T)    per 16 elements: the
//     product of the bare codes, scaled by the block's scale in float32;
//   O^T[16 elements][8 heads]  += V^T[16 x 16] (P s)^T    per 16 elements: the
//     scale of V goes into the probabilities (rounded to fp16).
// (Eight rows fill a sixteenth of a tcgen05 tile, and the operands would
// have to be widened into shared memory first.)  The cache's byte order gives
// each lane its fragments in 16-byte loads, free of bank conflicts; codes widen
// two at a time with one conversion.
//
// The online softmax keeps, per lane, a reference m that only moves (rescaling
// O) when a score exceeds it by 2^kSlack, so most records need no
// reduction over the warp.  Probabilities are formed as 2^(s - m + kShift):
// fp16's 11 bits then reach down to 2^-18 of the reference.
//
// Splits of a sequence leave their partials in the workspace; the CTA that
// takes the last ticket of a (sequence, kv head) merges them.  The number of
// splits that take part is that of the sequence's own length.
#include <math.h>

#include "g4_device.cuh"
#include "g4_internal.h"
#include "g4_kv4.cuh"

namespace g4 {
namespace {

constexpr int kHeads = 8;  // columns of the tensor-core product
constexpr float kSlack = 8.0f;
constexpr float kShift = 4.0f;
constexpr float kNoKey = -1e30f;  // reference of a state that has seen no key

template <int HD>
struct Kv4Cfg {
  static constexpr int NW = 4;                                  // warps per CTA
  static constexpr int GP = HD >= 256 ? 1 : 256 / HD;           // records per stage
  static constexpr int NST = 2;                                 // stages per warp
  static constexpr int MINB = HD >= 512 ? 2 : 4;                // CTAs per SM
  static constexpr int STAGE_B = GP * Kv4Rec<HD>::BYTES;
  static constexpr int RING_B = NW * NST * STAGE_B;
  static constexpr int MERGE_B = NW * kHeads * HD * 4;          // the warps' outputs
  static constexpr int AREA_B = RING_B > MERGE_B ? RING_B : MERGE_B;
  static constexpr int Q_OFF = AREA_B;                          // q fragments, fp16
  static constexpr int BAR_OFF = Q_OFF + kHeads * HD * 2;
  static constexpr int OK_OFF = BAR_OFF + NW * NST * 8;         // record present, per stage and record
  static constexpr int QF_OFF = OK_OFF + NW * NST * GP * 4;     // score factor of each head
  static constexpr int ML_OFF = QF_OFF + kHeads * 4;            // the warps' m and l
  static constexpr int W_OFF = ML_OFF + NW * kHeads * 8;        // merge weights
  static constexpr int SMEM_B = W_OFF + kHeads * kMaxSplits * 4;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 8 x 8 fp16 matrix held two elements per lane (row lane / 4), transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) { return as_u32(__floats2half2_rn(lo, hi)); }

template <int HD>
__global__ void __launch_bounds__(Kv4Cfg<HD>::NW * 32, Kv4Cfg<HD>::MINB)
    kv4_decode_kernel(const __grid_constant__ Kv4DecodeArgs a) {
  using C = Kv4Cfg<HD>;
  using R = Kv4Rec<HD>;
  constexpr int NW = C::NW, NST = C::NST, GP = C::GP, NB = HD / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  int* s_ok = reinterpret_cast<int*>(smem + C::OK_OFF);
  float* s_qf = reinterpret_cast<float*>(smem + C::QF_OFF);
  float* s_m = reinterpret_cast<float*>(smem + C::ML_OFF);
  float* s_l = s_m + NW * kHeads;
  float* s_w = reinterpret_cast<float*>(smem + C::W_OFF);
  __shared__ int s_last;

  const int split = blockIdx.x % a.nsplit;
  const int unit = blockIdx.x / a.nsplit;  // b * Hkv + kvh
  const int kvh = unit % a.Hkv, b = unit / a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = a.H / a.Hkv;
  uint64_t* wbar = bars + warp * NST;
  int* wok = s_ok + warp * NST * GP;
  if (lane == 0) {
    for (int i = 0; i < NST; ++i) mbar_init(smem_u32(&wbar[i]), 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_wait();
  pdl_trigger();

  const int L = min(max(a.lens[b], 0), a.len_cap);
  const int kbeg = a.window > 0 ? max(0, L - a.window) : 0;
  const int gfirst = kbeg >> 4, gend = (L + 15) >> 4;  // records of the visible keys
  const int nsplit = (gend - gfirst + a.chunk - 1) / a.chunk;  // splits that hold any
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (static_cast<size_t>(b) * a.H + kvh * G) * HD;
  if (split >= nsplit) {
    if (split == 0) {  // no key at all
      for (int i = threadIdx.x; i < G * HD / 2; i += NW * 32) reinterpret_cast<uint32_t*>(out)[i] = 0u;
    }
    return;
  }
  const int g0 = gfirst + split * a.chunk;
  const int ng = min(a.chunk, gend - g0);
  const int nstages = (ng + GP - 1) / GP;
  const int mine = nstages > warp ? (nstages - warp + NW - 1) / NW : 0;  // stages of this warp

  // Block ids of the warp's stages, 32 stages at a time: lane k % 32 holds
  // those of stage k and issues its copies.  The next 32 are loaded as soon as
  // the first of the current ones is used.
  const int32_t* row = a.table + static_cast<size_t>(b) * a.max_blocks;
  auto stage_group = [&](int k) { return g0 + (warp + k * NW) * GP; };
  int ids[GP], ids_next[GP];
  auto load_ids = [&](int window, int (&to)[GP]) {
    const int k = window * 32 + lane;
#pragma unroll
    for (int i = 0; i < GP; ++i) {
      const int gi = stage_group(k) + i;
      to[i] = -1;
      if (k < mine && gi < g0 + ng) {
        const int entry = gi >> (a.block_shift - 4);
        if (entry < a.max_blocks) to[i] = row[entry];
      }
    }
  };
  uint8_t* ring = smem + warp * (NST * C::STAGE_B);
  auto issue = [&](int k) {  // stage k of this warp into buffer k % NST
    if ((k & 31) == 0 && k > 0) {
#pragma unroll
      for (int i = 0; i < GP; ++i) ids[i] = ids_next[i];
      load_ids((k >> 5) + 1, ids_next);
    }
    if (lane == (k & 31)) {
      const int buf = k % NST;
      const uint32_t bar = smem_u32(&wbar[buf]);
      const uint32_t dst = smem_u32(ring + buf * C::STAGE_B);
      bool ok[GP];
      uint32_t bytes = 0;
#pragma unroll
      for (int i = 0; i < GP; ++i) {
        ok[i] = ids[i] >= 0 && ids[i] < a.n_blocks;
        wok[buf * GP + i] = ok[i];
        bytes += ok[i] ? R::BYTES : 0;
      }
      mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
      for (int i = 0; i < GP; ++i) {
        if (ok[i]) {
          const int in_block = (stage_group(k) + i) & ((1 << (a.block_shift - 4)) - 1);
          bulk_g2s(dst + i * R::BYTES, a.data + kv4_record<HD>(ids[i], kvh, in_block, a.Hkv, a.block_shift), R::BYTES,
                   bar);
        }
      }
    }
  };
  load_ids(0, ids);
  load_ids(1, ids_next);
  for (int k = 0; k < NST && k < mine; ++k) issue(k);

  // q fragments: lane (head g, t) holds elements 4t .. 4t+3 of every 16, two
  // blocks side by side; each head scaled by the power of two that brings its
  // largest element into [1, 2).
  {
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<size_t>(b) * a.H + kvh * G) * HD;
    for (int h = warp; h < kHeads; h += NW) {
      constexpr int PER = HD / 32;  // elements per lane, consecutive
      float x[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) x[i] = 0.0f;
      if (h < G) load_elems<PER>(q + h * HD + lane * PER, x);
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
      e = top > 0.0f ? min(max(e, -120), 120) : 0;
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      if (lane == 0) s_qf[h] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
      for (int i = 0; i < PER; i += 2) {
        const int d = lane * PER + i;
        const int blk = d >> 4, tt = (d >> 2) & 3;
        *reinterpret_cast<uint32_t*>(smem + C::Q_OFF + ((blk >> 1) * 32 + h * 4 + tt) * 16 + (blk & 1) * 8 + (d & 2) * 2) =
            pack_f16x2(x[i] * down, x[i + 1] * down);
      }
    }
  }
  __syncthreads();
  const float qf0 = s_qf[2 * t], qf1 = s_qf[2 * t + 1];

  float o[NB][4];
#pragma unroll
  for (int i = 0; i < NB; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
  float m0 = kNoKey, m1 = kNoKey, l0 = 0.0f, l1 = 0.0f;  // heads 2t and 2t + 1

  int done = 0;
  bool aborted = false;
  for (int k = 0; k < mine; ++k) {
    const int buf = k % NST;
    if (!warp_wait(smem_u32(&wbar[buf]), (k / NST) & 1, a.err)) {
      aborted = true;
      break;
    }
#pragma unroll 1
    for (int i = 0; i < GP; ++i) {
      const int gi = stage_group(k) + i;
      if (gi >= g0 + ng || !wok[buf * GP + i]) continue;
      const uint8_t* rec = ring + buf * C::STAGE_B + i * R::BYTES;
      const int pos0 = gi * kKv4Group;

      // S^T = K Q^T
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int p = 0; p < R::NP; ++p) {
        const uint4 kc = *reinterpret_cast<const uint4*>(rec + R::KC + p * 512 + lane * 16);
        const uint2 ks = *reinterpret_cast<const uint2*>(rec + R::KS + p * 64 + g * 8);
        const uint4 qa = *reinterpret_cast<const uint4*>(smem + C::Q_OFF + ((2 * p) * 32 + lane) * 16);
        const uint4 qb = *reinterpret_cast<const uint4*>(smem + C::Q_OFF + ((2 * p + 1) * 32 + lane) * 16);
        const uint32_t qw[8] = {qa.x, qa.y, qa.z, qa.w, qb.x, qb.y, qb.z, qb.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t w0 = w < 2 ? kc.x : kc.y, w1 = w < 2 ? kc.z : kc.w;
          const uint32_t sw = w < 2 ? ks.x : ks.y;
          float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          if (w & 1)
            mma_f16(d, e2m1x2_f16x2<2>(w0), e2m1x2_f16x2<2>(w1), e2m1x2_f16x2<3>(w0), e2m1x2_f16x2<3>(w1), qw[2 * w],
                    qw[2 * w + 1]);
          else
            mma_f16(d, e2m1x2_f16x2<0>(w0), e2m1x2_f16x2<0>(w1), e2m1x2_f16x2<1>(w0), e2m1x2_f16x2<1>(w1), qw[2 * w],
                    qw[2 * w + 1]);
          const float2 sc = __half22float2(as_half2(w & 1 ? e4m3x2_hi_f16x2(sw) : e4m3x2_f16x2(sw)));
          s[0] = fmaf(sc.x, d[0], s[0]);
          s[1] = fmaf(sc.x, d[1], s[1]);
          s[2] = fmaf(sc.y, d[2], s[2]);
          s[3] = fmaf(sc.y, d[3], s[3]);
        }
      }
      s[0] *= qf0;
      s[1] *= qf1;
      s[2] *= qf0;
      s[3] *= qf1;

      // Positions outside [kbeg, L): no weight, and their V scales (any bytes,
      // even NaN) read as zero.
      uint32_t vmask = 0xffffffffu;
      if (pos0 < kbeg || pos0 + kKv4Group > L) {
        auto seen = [&](int m) { return pos0 + m >= kbeg && pos0 + m < L; };
        if (!seen(g)) s[0] = s[1] = -INFINITY;
        if (!seen(g + 8)) s[2] = s[3] = -INFINITY;
        vmask = (seen(2 * t) ? 0xffu : 0u) | (seen(2 * t + 1) ? 0xff00u : 0u) | (seen(2 * t + 8) ? 0xff0000u : 0u) |
                (seen(2 * t + 9) ? 0xff000000u : 0u);
      }

      float top0 = fmaxf(s[0], s[2]), top1 = fmaxf(s[1], s[3]);
      if (__any_sync(0xffffffffu, top0 > m0 + kSlack || top1 > m1 + kSlack)) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, x));
          top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, x));
        }
        const float n0 = fmaxf(m0, top0), n1 = fmaxf(m1, top1);
        const float f0 = ex2_approx(m0 - n0), f1 = ex2_approx(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int x = 0; x < NB; ++x) {
          o[x][0] *= f0;
          o[x][1] *= f1;
          o[x][2] *= f0;
          o[x][3] *= f1;
        }
      }
      const float r0 = m0 - kShift, r1 = m1 - kShift;
      const float p0 = ex2_approx(s[0] - r0), p1 = ex2_approx(s[1] - r1);
      const float p2 = ex2_approx(s[2] - r0), p3 = ex2_approx(s[3] - r1);
      l0 += p0 + p2;
      l1 += p1 + p3;
      const __half2 pa = as_half2(transpose8x8(pack_f16x2(p0, p1)));  // head g, positions 2t, 2t+1
      const __half2 pb = as_half2(transpose8x8(pack_f16x2(p2, p3)));  // 2t+8, 2t+9

      // O^T += V^T (P s)^T
#pragma unroll
      for (int p = 0; p < R::NP; ++p) {
        const uint4 vc = *reinterpret_cast<const uint4*>(rec + R::VC + p * 512 + lane * 16);
        const uint4 vs = *reinterpret_cast<const uint4*>(rec + R::VS + p * 64 + t * 16);
        // pairs of positions side by side, for the even and the odd elements
        const uint32_t lo01 = (vc.x & 0x0f0f0f0fu) | ((vc.y << 4) & 0xf0f0f0f0u);
        const uint32_t hi01 = ((vc.x >> 4) & 0x0f0f0f0fu) | (vc.y & 0xf0f0f0f0u);
        const uint32_t lo23 = (vc.z & 0x0f0f0f0fu) | ((vc.w << 4) & 0xf0f0f0f0u);
        const uint32_t hi23 = ((vc.z >> 4) & 0x0f0f0f0fu) | (vc.w & 0xf0f0f0f0u);
        const uint32_t vsw[4] = {vs.x & vmask, vs.y & vmask, vs.z & vmask, vs.w & vmask};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t b0 = as_u32(__hmul2(pa, as_half2(e4m3x2_f16x2(vsw[w]))));
          const uint32_t b1 = as_u32(__hmul2(pb, as_half2(e4m3x2_hi_f16x2(vsw[w]))));
          float(&d)[4] = o[4 * p + w];
          switch (w) {
            case 0: mma_f16(d, e2m1x2_f16x2<0>(lo01), e2m1x2_f16x2<0>(hi01), e2m1x2_f16x2<0>(lo23), e2m1x2_f16x2<0>(hi23), b0, b1); break;
            case 1: mma_f16(d, e2m1x2_f16x2<1>(lo01), e2m1x2_f16x2<1>(hi01), e2m1x2_f16x2<1>(lo23), e2m1x2_f16x2<1>(hi23), b0, b1); break;
            case 2: mma_f16(d, e2m1x2_f16x2<2>(lo01), e2m1x2_f16x2<2>(hi01), e2m1x2_f16x2<2>(lo23), e2m1x2_f16x2<2>(hi23), b0, b1); break;
            default: mma_f16(d, e2m1x2_f16x2<3>(lo01), e2m1x2_f16x2<3>(hi01), e2m1x2_f16x2<3>(lo23), e2m1x2_f16x2<3>(hi23), b0, b1); break;
          }
        }
      }
    }
    __syncwarp();  // every lane is done with the stage
    done = k + 1;
    if (k + NST < mine) issue(k + NST);
  }
  if (aborted) {  // copies of this warp still in flight
    for (int k = done; k < mine && k < done + NST; ++k) warp_wait(smem_u32(&wbar[k % NST]), (k / NST) & 1, nullptr);
  }

  // The warps' states through shared memory (the rings are free now).
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, x);
    l1 += __shfl_xor_sync(0xffffffffu, l1, x);
  }
  if (g == 0) {
    s_m[warp * kHeads + 2 * t] = m0;
    s_m[warp * kHeads + 2 * t + 1] = m1;
    s_l[warp * kHeads + 2 * t] = l0;
    s_l[warp * kHeads + 2 * t + 1] = l1;
  }
  __syncthreads();
  float M0 = s_m[2 * t], M1 = s_m[2 * t + 1];
#pragma unroll
  for (int w = 1; w < NW; ++w) {
    M0 = fmaxf(M0, s_m[w * kHeads + 2 * t]);
    M1 = fmaxf(M1, s_m[w * kHeads + 2 * t + 1]);
  }
  const float f0 = ex2_approx(m0 - M0), f1 = ex2_approx(m1 - M1);
  float* os = reinterpret_cast<float*>(smem) + warp * kHeads * HD;
#pragma unroll
  for (int x = 0; x < NB; ++x) {
    const int d = x * 16 + 2 * g;
    if (2 * t < G) *reinterpret_cast<float2*>(os + (2 * t) * HD + d) = make_float2(o[x][0] * f0, o[x][2] * f0);
    if (2 * t + 1 < G) *reinterpret_cast<float2*>(os + (2 * t + 1) * HD + d) = make_float2(o[x][1] * f1, o[x][3] * f1);
  }
  __syncthreads();
  const size_t pbase = (static_cast<size_t>(b) * a.H + kvh * G) * a.nsplit;
  for (int idx = threadIdx.x; idx < G * HD / 4; idx += NW * 32) {
    const int h = idx * 4 / HD, d = idx * 4 % HD;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float M = kNoKey, l = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) + (w * kHeads + h) * HD + d);
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
      M = fmaxf(M, s_m[w * kHeads + h]);
    }
#pragma unroll
    for (int w = 0; w < NW; ++w) l += s_l[w * kHeads + h] * ex2_approx(s_m[w * kHeads + h] - M);
    if (nsplit == 1) {
      // (l is zero only where no key was present; a NaN stays one)
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const float f[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
      store_elems<4>(out + h * HD + d, f);
    } else {
      const size_t pr = pbase + static_cast<size_t>(h) * a.nsplit + split;
      *reinterpret_cast<float4*>(a.ws_o + pr * HD + d) = acc;
      if (d == 0) {
        a.ws_m[pr] = M;
        a.ws_l[pr] = l;
      }
    }
  }
  if (nsplit == 1) return;

  __threadfence();
  __syncthreads();
  unsigned* ticket = a.tickets + unit;
  if (threadIdx.x == 0) s_last = atomicAdd(ticket, 1u) == static_cast<unsigned>(nsplit - 1);
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int h = warp; h < G; h += NW) {
    const size_t p0 = pbase + static_cast<size_t>(h) * a.nsplit;
    float M = kNoKey;
    for (int i = lane; i < nsplit; i += 32) M = fmaxf(M, __ldcg(a.ws_m + p0 + i));
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    float l = 0.0f;
    for (int i = lane; i < nsplit; i += 32) {
      const float w = ex2_approx(__ldcg(a.ws_m + p0 + i) - M);
      s_w[h * kMaxSplits + i] = w;
      l += w * __ldcg(a.ws_l + p0 + i);
    }
    l = warp_sum(l);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    __syncwarp();
    for (int i = lane; i < nsplit; i += 32) s_w[h * kMaxSplits + i] *= inv;
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < G * HD / 4; idx += NW * 32) {
    const int h = idx * 4 / HD, d = idx * 4 % HD;
    const float* src = a.ws_o + (pbase + static_cast<size_t>(h) * a.nsplit) * HD + d;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int i = 0; i < nsplit; ++i) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(src + static_cast<size_t>(i) * HD));
      const float w = s_w[h * kMaxSplits + i];
      acc[0] = fmaf(w, v.x, acc[0]);
      acc[1] = fmaf(w, v.y, acc[1]);
      acc[2] = fmaf(w, v.z, acc[2]);
      acc[3] = fmaf(w, v.w, acc[3]);
    }
    store_elems<4>(out + h * HD + d, acc);
  }
  if (threadIdx.x == 0) *ticket = 0u;  // ready for the next call
}

template <int HD>
cudaError_t launch_h(const Kv4DecodeArgs& a, cudaStream_t s) {
  using C = Kv4Cfg<HD>;
  const cudaError_t e = set_smem_limit_once<kv4_decode_kernel<HD>>(C::SMEM_B);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(a.B) * a.Hkv * a.nsplit));
  cfg.blockDim = dim3(C::NW * 32);
  cfg.dynamicSmemBytes = C::SMEM_B;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_decode_kernel<HD>, a);
}

}  // namespace

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, cudaStream_t s) {
  switch (a.hd) {
    case 64: return launch_h<64>(a, s);
    case 128: return launch_h<128>(a, s);
    case 256: return launch_h<256>(a, s);
    case 512: return launch_h<512>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

Kv4DecodePlan kv4_decode_plan(int window, int hd, int H, int Hkv, int B, int max_seq_len) {
  Kv4DecodePlan p;
  const int span = window > 0 && window < max_seq_len ? window : max_seq_len;
  // a window that starts inside a record touches one more
  const int groups = static_cast<int>((static_cast<long long>(span) + 15) / 16) + (span < max_seq_len ? 1 : 0);
  const long long units = static_cast<long long>(B) * Hkv;
  const int slots = sm_count() * (hd >= 512 ? 2 : 4);
  // Two waves of CTAs even out ragged lengths; a split has at least two
  // records per warp.
  long long want = (2LL * slots + units - 1) / units;
  const int most = (groups + 7) / 8;
  if (want > most) want = most;
  if (want > kMaxSplits) want = kMaxSplits;
  if (want < 1) want = 1;
  p.chunk = static_cast<int>((groups + want - 1) / want);
  p.nsplit = (groups + p.chunk - 1) / p.chunk;
  if (p.nsplit <= 1) {
    p.o_bytes = p.m_bytes = p.t_bytes = p.ws_bytes = 0;
  } else {
    const size_t np = static_cast<size_t>(B) * H * p.nsplit;
    p.o_bytes = (np * hd * 4 + 255) / 256 * 256;
    p.m_bytes = (np * 4 + 255) / 256 * 256;
    p.t_bytes = (static_cast<size_t>(units) * 4 + 255) / 256 * 256;
    p.ws_bytes = p.o_bytes + 2 * p.m_bytes + p.t_bytes;
  }
  return p;
}

}  // namespace g4
