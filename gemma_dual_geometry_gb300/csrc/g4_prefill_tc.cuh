// Step a5 in bf16: causal GQA flash attention on the tcgen05 tensor cores.
//
// Semantics as in g4_attn_simt.cuh (cortiq-engine g4e.rs `attend_all_heads`
// with scale 1.0 and the sliding window, ferrox-models gemma4_engine.rs
// `causal_gqa_attention[_windowed]`): o_i = sum_j softmax_j(scale q_i.k_j) v_j
// over keys j <= i (and i - j < window on sliding layers), query head h
// reading kv head h / (H / Hkv).
//
// The BIDIR instantiation is the encoder form (taconite-embeddinggemma2
// model.rs `text_attention`): the T tokens of a sequence are both queries
// and keys (cache rows 0..T-1), with no causal mask, and key j is visible
// from query i iff |i - j| <= window on a sliding layer.  Only the tile
// range of a work item and the visible interval of a row differ.  On a
// sliding-window ring cache (max_len rows, a multiple of the 128-key tile)
// key position p is row p mod max_len; the masks stay in positions.
//
// The MODS instantiations modify the scores (g4_attn_prefill_mods); they are
// compiled in g4_prefill_mods.cu, whose comment says what differs.
//
// A work item is a 128-query-row tile of one (sequence, head) and, for
// head_dim 512, one 256-wide half of the output columns (two items per tile
// then recompute the same scores; TMEM holds 512 f32 columns per SM and a
// 128 x 512 accumulator alone would fill it).  Items run in (sequence, kv
// head) groups, heaviest query tiles first, so the CTAs in flight share their
// K / V in L2.  The kernel is persistent: one CTA per SM takes items one
// after another from a global counter (the producer draws them and passes
// them on through a 4-entry queue in shared memory), with its barriers, ring and TMEM
// running on from item to item, so the next item's Q and first K parts load
// while the current one finishes.  Warp roles (320 threads, MODS 608):
//   warp 0      TMA producer (converged; one elected lane issues): the Q
//               tile, then K parts (128 keys x 64..256 dims) and V parts
//               (64..128 keys x DV dims) as 5-D boxes, one request per
//               32-64 KB (a request costs the SM about the same whatever its
//               size), through a ring of slots, 128-byte swizzled.
//   warp 1      allocates TMEM and runs the MMA issue loop converged; one
//               elected lane issues every tcgen05.mma from precomputed
//               descriptors:
//                 S[j%2] = Q K_j^T      (M=128, N=128, K=head_dim; A, B from
//                                        shared memory, K-major)
//                 O     += P_j V_j      (M=128, N=DV,  K=128; A = P_j from
//                                        TMEM, B = V_j MN-major)
//               in the order QK_0, QK_1, PV_0, QK_2, PV_1, ... so the score
//               MMA of the next tile overlaps the softmax of this one.
//   warps 2-9   softmax (MODS: 2-17, quarters of a row instead of halves):
//               two warps per TMEM lane quarter (a warp may only touch its quarter's 32 lanes), each thread half a query row
//               (64 of the 128 score columns; TMEM lane = row): load the
//               whole S row with tcgen05.ld (both threads of a row find the
//               same maximum), mask (one visible key interval per row:
//               causal end, window start, keys past the cache), online
//               softmax in the log2 domain with the running maximum raised
//               only when it grows by more than 2^64 (the stale maximum is
//               exact for O / l), rescale its half of the O row in TMEM when
//               it is raised, and write its P half as bf16 over the S buffer
//               (packed: 32 columns), once the other warp of the quarter has
//               read the row too (P lands on S columns both warps read).
//               The row sum l adds the bf16-rounded P
//               values, the weights the PV MMA really applies, so a row
//               dominated by one key returns that key's value without the
//               rounding error of P; the two halves' sums meet in shared
//               memory once, at the end.  Epilogue: O / l as bf16 into the
//               ring slots of the item's last V parts (swizzled like the
//               output tensor map), TMA stores, then those slots are freed.
//   warp 18     (MODS) the TMA stores of staged outputs, after which it frees their
//               slots; the softmax warps go on with the next item meanwhile.
// TMEM columns: S0/P0 [0,128), S1/P1 [128,256), O [256, 256 + DV).
// The MMAs of one thread execute in issue order, so QK_{j+2} (issued after
// PV_j) overwrites P_j only after PV_j has read it; no barrier is needed
// between them.  Barriers come in pairs indexed by tile parity (j % 2), which
// keeps each phase unambiguous for waiters that skip phases.
// Key tiles wholly outside every row's band are never loaded.
#pragma once

#include <math.h>

#include <type_traits>

#include "g4_device.cuh"
#include "g4_internal.h"
#include "g4_tiles.h"

namespace g4 {
namespace {

// What an instantiation computes: causal attention, the encoder's, or attention with modified scores.
constexpr int kCausal = 0, kBidir = 1, kMods = 2;

constexpr int kBM = 128;       // query rows per CTA
constexpr int kBN = 128;       // keys per tile
constexpr int kChunkB = 16384;  // 128 rows x 64 bf16, one 128-byte-swizzled block
// Softmax warps, beside the producer and the MMA issuer.  MODS: twice as many, each thread a quarter of a row, and a
// warp that stores the output.
template <int MODE>
constexpr int kSoftWarps = MODE == kMods ? 16 : 8;
template <int MODE>
constexpr int kThreads = 64 + 32 * kSoftWarps<MODE> + (MODE == kMods ? 32 : 0);
constexpr int kModsParts = kSoftWarps<kMods> / 4;  // parts of a row's columns
constexpr int kMaxSlots = 12;
constexpr int kSmemMax = 232448;  // opt-in shared memory per block
// The exponent base of a row is raised only when a tile's maximum exceeds it
// by more than 2^64: P <= 2^64 in bf16 and O <= 2^64 * keys * |v| in f32 stay
// far from overflow, and rescaling O (a TMEM round trip) becomes rare.
constexpr float kRescaleLog2 = 64.0f;

template <int HD>
struct TcCfg {
  static constexpr int DV = HD < 256 ? HD : 256;  // output columns per CTA
  static constexpr int NDH = HD / DV;             // CTAs per (tile, head)
  static constexpr int QCH = HD / 64;             // 64-dim chunks of Q and of a K tile
  // A TMA request costs the SM about 576 cycles whatever its size up to
  // 32 KB (64 KB: ~900), so tiles move as few large multi-dimensional boxes:
  // a K part is 128 keys x CPP 64-dim chunks, a V part VKP keys x DV dims.
  static constexpr int KPARTS = HD == 512 ? 4 : 1;
  static constexpr int CPP = QCH / KPARTS;          // 64-dim chunks per K part
  static constexpr int KPB = CPP * kChunkB;         // K part bytes
  static constexpr int VKP = HD == 512 ? 64 : 128;  // keys per V part
  static constexpr int VPARTS = kBN / VKP;
  static constexpr int VPB = VKP * DV * 2;          // V part bytes
  static constexpr int SLOTB = KPB > VPB ? KPB : VPB;
  // The output tile (DV / 64 chunks) is staged in the slots of the last V
  // parts of the item: CPS chunks per slot, OSLOTS slots.
  static constexpr int CPS = SLOTB / kChunkB;
  static constexpr int OSLOTS = (DV / 64) / CPS;
  static constexpr int Q_OFF = 0;
  static constexpr int RING_OFF = Q_OFF + QCH * kChunkB;
  static constexpr int BAR_B = 3 * 1024;
  static constexpr int NSLOT_FIT = (kSmemMax - BAR_B - RING_OFF) / SLOTB;
  static constexpr int NSLOT = NSLOT_FIT < kMaxSlots ? NSLOT_FIT : kMaxSlots;
  static constexpr int BAR_OFF = RING_OFF + NSLOT * SLOTB;
  static constexpr int SMEM_B = BAR_OFF + BAR_B;
  static_assert(NSLOT >= 2, "ring depth");
  static_assert(SMEM_B <= kSmemMax, "shared memory budget");
  static_assert(VKP % 16 == 0 && kBN % VKP == 0 && QCH % KPARTS == 0, "tiling");
  static_assert(SLOTB % kChunkB == 0 && (DV / 64) % CPS == 0 && OSLOTS >= 1 && OSLOTS <= VPARTS &&
                    OSLOTS < NSLOT && VPB == SLOTB,
                "output staging in the ring");
};

struct TcBars {
  uint64_t q_full;     // the current item's Q tile has landed (one phase per item)
  uint64_t q_free;     // every QK MMA of the current item is complete (Q may be replaced)
  uint64_t s_full[2];  // QK_j complete (tile parity)
  uint64_t p_full[2];  // P_j written to TMEM by all softmax threads
  uint64_t o_done[2];  // PV_j complete
  uint64_t drain;
  uint64_t sum_full[4];  // [lane quarter]: both row-sum shares written
  uint64_t s_read[4];    // [lane quarter]: its warps have S_j in registers (P_j may overwrite it)
  // MODS:
  uint64_t x_full[4];    // [lane quarter]: its warps have written their parts of an exchange
  uint64_t x_free[4];    // [lane quarter]: and read those of all
  uint64_t o_staged;     // the item's output is in its ring slots
  uint64_t o_taken;      // the storing warp has seen that
  uint64_t full[kMaxSlots];
  uint64_t empty[kMaxSlots];
  uint64_t it_full[4];   // work-item queue entry written (by the producer)
  uint64_t it_empty[4];  // entry read by the MMA issuer and the softmax warps (MODS: each of them, and the storing warp)
  int items[4];          // work-item queue: item index, or -1 when none is left
  int kbeg[4], kend[4];  // MODS: the keys that some row of the item sees, [kbeg, kend)
  uint32_t tmem_base;
  int abort;
  // MODS: [tile parity][lane quarter][part]: number of the tile whose maximum it wants raised
  alignas(16) int raise[2][4][kModsParts];
  float red[kModsParts][kBM];   // [part of the columns][row]: row-sum shares; MODS: row maxima too
};
static_assert(sizeof(TcBars) <= TcCfg<64>::BAR_B, "barrier block");

// All 256 softmax threads meet (named barrier 1) and learn whether any of
// them passed a nonzero flag.
__device__ __forceinline__ bool softmax_sync_any(int flag) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 q, %1, 0;\n\t"
      "bar.red.or.pred p, 1, 256, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(any)
      : "r"(flag)
      : "memory");
  return any != 0;
}

template <int MODE>
using TcArgsOf = std::conditional_t<MODE == kMods, ModsTcArgs, PrefillTcArgs>;

// Work item -> (output half, q head of the group, q tile, kv head, sequence)
// and the key tiles it needs.  Items run in (sequence, kv head) groups so the
// CTAs working at the same time share one K / V in L2; within a group the
// heaviest (last) query tiles come first.
struct TcItem {
  int dh, h, kvh, b;
  int q0, valid_rows, qpos_first, Lk, kt_begin, ntiles;
  int kbeg;  // MODS only: the first key that some row sees (Lk: one past the last one)
};

// MODS: the interval of keys that row r of the item sees (empty: 0, 0).
__device__ __forceinline__ int2 tc_row_keys(const ModsTcArgs& a, const TcItem& w, int r) {
  if (r >= w.valid_rows) return make_int2(0, 0);
  const int q_start = min(max(a.q_start[w.b], 0), 0x7fffffff - a.T);
  const int held = a.ring ? q_start + a.T : min(q_start + a.T, a.max_len);
  const int pos = q_start + w.q0 + r;
  const size_t tok = static_cast<size_t>(w.b) * a.T + w.q0 + r;
  int lo = a.sliding ? pos - a.window + 1 : 0, hi = pos + 1;
  if (a.key_begin != nullptr) lo = a.key_begin[tok];
  if (a.key_end != nullptr) hi = a.key_end[tok];
  lo = max(lo, a.ring ? max(0, held - a.max_len) : 0);
  hi = min(hi, held);
  return lo < hi ? make_int2(lo, hi) : make_int2(0, 0);  // (ends from -2^31 on do not come into any difference)
}

// MODS: the keys of an item, known to the producer that drew it.
__device__ __forceinline__ void tc_set_keys(TcItem& w, int kbeg, int kend) {
  w.kbeg = kbeg;
  w.Lk = kend;
  w.kt_begin = kbeg / kBN;
  w.ntiles = kend > kbeg ? tiles_before(kend, kBN) - w.kt_begin : 0;
}

template <int NDH, int MODE, typename Args>
__device__ __forceinline__ TcItem tc_item(const Args& a, int it, int nqt) {
  constexpr bool BIDIR = MODE == kBidir;
  TcItem w;
  const int grp = a.H / a.Hkv;
  int idx = it;
  w.dh = idx % NDH;
  idx /= NDH;
  const int hq = idx % grp;
  idx /= grp;
  const int qt = nqt - 1 - idx % nqt;
  idx /= nqt;
  w.kvh = idx % a.Hkv;
  w.b = idx / a.Hkv;
  w.h = w.kvh * grp + hq;
  w.q0 = qt * kBM;
  w.valid_rows = min(kBM, a.T - w.q0);
  if constexpr (MODE == kMods) {
    w.qpos_first = min(max(a.q_start[w.b], 0), 0x7fffffff - a.T) + w.q0;
    w.Lk = w.kt_begin = w.ntiles = w.kbeg = 0;  // (tc_set_keys)
    return w;
  }
  const int q_start = BIDIR ? 0 : a.q_start[w.b];
  w.qpos_first = q_start + w.q0;
  const int qpos_last = w.qpos_first + w.valid_rows - 1;
  int kbeg, kend;
  if constexpr (BIDIR) {
    // Encoder: the sequence's own T keys, no causal mask; query i sees
    // [i - window, i + window] on a sliding layer (window <= T here).
    w.Lk = a.T;
    kbeg = a.sliding ? max(0, w.qpos_first - a.window) : 0;
    kend = a.sliding ? min(qpos_last + a.window + 1, w.Lk) : w.Lk;
  } else {
    // keys held: positions [0, Lk) (a ring holds the last max_len of them)
    w.Lk = a.ring ? q_start + a.T : min(q_start + a.T, a.max_len);
    kend = min(qpos_last + 1, w.Lk);
    kbeg = a.sliding ? max(0, w.qpos_first - a.window + 1) : 0;
  }
  w.kt_begin = kbeg / kBN;
  w.ntiles = max(0, tiles_before(kend, kBN) - w.kt_begin);
  return w;
}

// ---------------------------------------------------------------- MODS: softmax and output

// Arrives for the warp once all of its lanes have come here.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(bar));
}

__device__ __forceinline__ int4 ld_shared_int4(uint32_t addr) {
  int4 v;
  asm volatile("ld.volatile.shared.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// The smaller one; NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Raw scores q.k of N keys become c tanh(s / c) in log2 units, with tanh(y) = 1 - 2 / (1 + e^2y), off by about 2^-22.
// Four reciprocals are one of their product: a reciprocal takes the special-function unit as long as two exponentials
// (capping costs a tile of 128 keys 970 cycles, 1430 with a reciprocal each).  e^2y is cut off at 2^30, where the tanh
// is 1 in float32, so that the product stays finite; a NaN makes its neighbours NaN, which are the same row's.
template <int N>
__device__ __forceinline__ void cap_scores(float (&s)[N], float cap_in, float cap_log2) {
  const float2 in2 = make_float2(cap_in, cap_in), one = make_float2(1.0f, 1.0f), cap2 = make_float2(cap_log2, cap_log2);
  const float2 twice = make_float2(-2.0f * cap_log2, -2.0f * cap_log2);
#pragma unroll
  for (int n = 0; n < N; n += 4) {
    const float2 x = __fmul2_rn(make_float2(s[n], s[n + 1]), in2), y = __fmul2_rn(make_float2(s[n + 2], s[n + 3]), in2);
    const float2 d = __fadd2_rn(make_float2(ex2_approx(min_nan(x.x, 30.0f)), ex2_approx(min_nan(x.y, 30.0f))), one);
    const float2 e = __fadd2_rn(make_float2(ex2_approx(min_nan(y.x, 30.0f)), ex2_approx(min_nan(y.y, 30.0f))), one);
    const float de = d.x * d.y, ee = e.x * e.y;
    const float r = rcp_approx(de * ee);
    const float rd = r * ee, re = r * de;  // 1 / (d.x d.y), 1 / (e.x e.y)
    const float2 a = __ffma2_rn(__fmul2_rn(make_float2(rd, rd), make_float2(d.y, d.x)), twice, cap2);
    const float2 b = __ffma2_rn(__fmul2_rn(make_float2(re, re), make_float2(e.y, e.x)), twice, cap2);
    s[n] = a.x;
    s[n + 1] = a.y;
    s[n + 2] = b.x;
    s[n + 3] = b.y;
  }
}

// One row's output in NC columns again, without the tensor cores, where a key that the row does not see holds a NaN or
// an infinity (its weight is zero, but zero times that is a NaN in the product): the warp forms the weights of the keys
// that it does see, several at a time, with the row's own base m, and adds their values up, two columns per lane.
// inv_l: 1 / row sum.  Done once all columns are NaN: the row sees one itself.
//   A warp has up to 32 such rows (of 16384 keys 307 ms at head_dim 512, 158 at 128; with all CTAs at it, up to two items
// each, 449 and 152), and the others' bounded waits go on meanwhile, so rows of more than kAgainKeys keys are left as they are.
constexpr int kAgainKeys = 1 << 15;

template <int HD, int NC>
__device__ __noinline__ float2 row_again(const ModsTcArgs& a, int b, int h, int tok, int2 keys, int qpos, float slope,
                                         float m, float inv_l, int col0) {
  constexpr int KB = HD < 256 ? 8 : 4;  // keys at a time
  constexpr int W = HD / 64 < 4 ? HD / 64 : 4;  // 32-bit words of a row that a lane loads at once
  constexpr int NW = HD / 64 / W;
  const int lane = threadIdx.x & 31;
  const int kvh = h / (a.H / a.Hkv);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + ((static_cast<size_t>(b) * a.T + tok) * a.H + h) * HD;
  const __nv_bfloat16* ck = static_cast<const __nv_bfloat16*>(a.ck);
  const __nv_bfloat16* cv = static_cast<const __nv_bfloat16*>(a.cv) + col0;
  const size_t head = (static_cast<size_t>(b) * a.Hkv + kvh) * a.max_len;
  auto load = [&](const __nv_bfloat16* row, int n, uint32_t (&x)[W]) {
    const __nv_bfloat16* from = row + (n * 32 + lane) * 2 * W;
    if constexpr (W == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(from);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else if constexpr (W == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(from);
      x[0] = v.x; x[1] = v.y;
    } else {
      x[0] = *reinterpret_cast<const uint32_t*>(from);
    }
  };
  float2 o = make_float2(0.0f, 0.0f);
  // (keys are counted from the row's first one: past the last one there may be no position)
  const int nkeys = keys.y - keys.x;
#pragma unroll 1
  for (int j0 = 0; j0 < nkeys; j0 += KB) {
    size_t row[KB];
    float s[KB];
    uint32_t v[KB];
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int j = keys.x + min(j0 + i, nkeys - 1);
      row[i] = (head + (a.ring ? j % a.max_len : j)) * HD;
      s[i] = 0.0f;
      v[i] = lane * 2 < NC ? *reinterpret_cast<const uint32_t*>(cv + row[i] + lane * 2) : 0u;
    }
#pragma unroll 1
    for (int n = 0; n < NW; ++n) {
      uint32_t x[W], y[KB][W];
      load(q, n, x);
#pragma unroll
      for (int i = 0; i < KB; ++i) load(ck + row[i], n, y[i]);
#pragma unroll
      for (int i = 0; i < KB; ++i)
#pragma unroll
        for (int w = 0; w < W; ++w) s[i] = fmaf(bf16_lo(x[w]), bf16_lo(y[i][w]), fmaf(bf16_hi(x[w]), bf16_hi(y[i][w]), s[i]));
    }
#pragma unroll
    for (int i = 0; i < KB; ++i) s[i] = warp_sum(s[i]);
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      float t = s[i] * a.scale_log2;
      if (a.cap_log2 > 0.0f)
        t = fmaf(-2.0f * a.cap_log2, rcp_approx(1.0f + ex2_approx(min_nan(s[i] * a.cap_in, 30.0f))), a.cap_log2);
      t = fmaf(-slope, fabsf(static_cast<float>(qpos - keys.x - (j0 + i))), t);
      const float p = bf16_lo(pack_bf16x2(ex2_approx(t - m), 0.0f));
      if (j0 + i < nkeys) {
        o.x = fmaf(p, bf16_lo(v[i]), o.x);
        o.y = fmaf(p, bf16_hi(v[i]), o.y);
      }
    }
    if (__all_sync(0xffffffffu, lane * 2 >= NC || (o.x != o.x && o.y != o.y))) break;
  }
  return make_float2(o.x * inv_l, o.y * inv_l);
}

// The softmax warps' work (16 warps; lane r of a quarter holds a row, four warps a quarter of its columns each).
//   Item by item and tile by tile as in the causal kernel, from the last key tile to the first: a distance bias falls
// from the diagonal on, so that the first tile's maximum is the largest and O need not be rescaled
// (2 x 4096 tokens of head_dim 128 took 15 % longer in ascending order).
//   A row's exponent base only has to be common to its parts and within 2^64 of the running maximum, so parts that
// find their own maxima no further above the base go on without asking the others: the wish to raise the base
// travels with the barrier that they need anyway, before P_j overwrites S_j, and only then do they exchange maxima.
template <int HD, bool CAP, bool BIAS>
__device__ __forceinline__ void softmax_mods(const ModsTcArgs& a, TcBars* bars, uint32_t tmem, uint32_t sRing, int nqt) {
  using C = TcCfg<HD>;
  constexpr int N = kBN / kModsParts;           // score columns per thread
  constexpr int kDVP = C::DV / kModsParts;      // O columns per thread
  constexpr int kCW = kDVP < 32 ? kDVP : 32;    // of which so many are loaded at once
  constexpr int kParts = C::KPARTS + C::VPARTS;  // ring parts per key tile
  static_assert(N == 32, "a part of S is one load");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;       // TMEM lane quarter this warp may access
  const int part = (warp - 2) >> 2;   // which quarter of the columns
  const int r = quarter * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t tmem_O = tmem + 256 + lane_off + part * kDVP;
  volatile int* abort = &bars->abort;

  // All four parts of a row learn each other's number.
  int xc = 0;
  auto exchange = [&](float v, float (&all)[kModsParts]) -> bool {
    if (xc > 0 && !warp_wait(smem_u32(&bars->x_free[quarter]), (xc - 1) & 1, a.err, abort)) return false;
    bars->red[part][r] = v;
    warp_arrive(&bars->x_full[quarter]);
    if (!warp_wait(smem_u32(&bars->x_full[quarter]), xc & 1, a.err, abort)) return false;
#pragma unroll
    for (int i = 0; i < kModsParts; ++i) all[i] = bars->red[i][r];
    warp_arrive(&bars->x_free[quarter]);
    ++xc;
    return true;
  };

  // Item n of the queue, with this row's keys and slope; false: none is left, or a wait gave up.
  struct Next {
    int qpos;             // the row's position
    int kt_last, ntiles;  // the last key tile and how many there are
    int2 keys;
    float slope;
    int it;
  };
  auto fetch = [&](int n, Next& x) -> bool {
    const int e = n & 3;
    if (!warp_wait(smem_u32(&bars->it_full[e]), (n >> 2) & 1, a.err, abort)) return false;
    const int it = *reinterpret_cast<volatile int*>(&bars->items[e]);
    const int kbeg = *reinterpret_cast<volatile int*>(&bars->kbeg[e]);
    const int kend = *reinterpret_cast<volatile int*>(&bars->kend[e]);
    warp_arrive(&bars->it_empty[e]);
    if (it < 0) return false;
    TcItem w = tc_item<C::NDH, kMods>(a, it, nqt);
    tc_set_keys(w, kbeg, kend);
    x.qpos = w.qpos_first + min(r, w.valid_rows - 1);
    x.kt_last = w.kt_begin + w.ntiles - 1;
    x.ntiles = w.ntiles;
    x.keys = tc_row_keys(a, w, r);
    x.slope = BIAS ? a.slopes[w.h] * 1.4426950408889634f : 0.0f;
    x.it = it;
    return true;
  };

  int J = 0;      // tiles of earlier items
  int nq = 0;     // items done that had any
  int parts = 0;  // ring parts of earlier items
  Next cur;
  bool ok = fetch(0, cur);
  for (int n = 0; ok; ++n) {
    const int ntiles = cur.ntiles;
    if (ntiles == 0) {
      // no row sees a key
      const TcItem w = tc_item<C::NDH, kMods>(a, cur.it, nqt);
      if (r < w.valid_rows) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) +
                             (((static_cast<size_t>(w.b) * a.T + w.q0 + r) * a.H + w.h) * HD + w.dh * C::DV + part * kDVP);
#pragma unroll
        for (int i = 0; i < kDVP / 8; ++i) reinterpret_cast<uint4*>(dst)[i] = make_uint4(0, 0, 0, 0);
      }
      ok = fetch(n + 1, cur);
      continue;
    }
    float m = -INFINITY;  // exponent base in log2 units
    float l = 0.0f;       // this part's share of the row sum
    for (int j = 0; j < ntiles; ++j) {
      const int sb = (J + j) & 1;
      if (!warp_wait(smem_u32(&bars->s_full[sb]), ((J + j) >> 1) & 1, a.err, abort)) { ok = false; break; }
      tc_fence_after();
      float s[N];
      {
        uint32_t raw[N];
        tmem_ld32(tmem + lane_off + sb * kBN + part * N, raw);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = __uint_as_float(raw[i]);
      }
      const int k0 = (cur.kt_last - j) * kBN + part * N;  // this part's first key
      const int lo = max(cur.keys.x - k0, 0), hi = min(cur.keys.y - k0, N);
      const bool masked = lo > 0 || hi < N;
      // bit i: key k0 + i is seen
      const uint32_t seen = lo < hi ? (0xffffffffu << lo) & (0xffffffffu >> (N - hi)) : 0u;
      if constexpr (CAP) {
        if (masked) {  // (what nobody sees may be NaN)
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (!(seen >> i & 1)) s[i] = 0.0f;
        }
        cap_scores(s, a.cap_in, a.cap_log2);
      }
      const float c2 = CAP ? 1.0f : a.scale_log2;
      if constexpr (BIAS) {
        const float slope = cur.slope, apart = static_cast<float>(cur.qpos - k0);
        if (cur.qpos - k0 >= N - 1) {
          // all keys at or before the query: c2 s - slope apart + slope i
          const float2 c22 = make_float2(c2, c2), off = make_float2(-slope * apart, -slope * apart);
          const float2 sl2 = make_float2(slope, slope);
#pragma unroll
          for (int i = 0; i < N; i += 2) {
            float2 t = __ffma2_rn(make_float2(s[i], s[i + 1]), c22, off);
            t = __ffma2_rn(sl2, make_float2(static_cast<float>(i), static_cast<float>(i + 1)), t);
            s[i] = t.x;
            s[i + 1] = t.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) s[i] = fmaf(-slope, fabsf(apart - static_cast<float>(i)), s[i] * c2);
        }
      }
      if (masked) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (!(seen >> i & 1)) s[i] = -INFINITY;
      }
      const float c3 = BIAS ? 1.0f : c2;  // what the scores are still multiplied by
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < N; i += 2) mx[i / 2 & 3] = fmaxf(mx[i / 2 & 3], fmaxf(s[i], s[i + 1]));
      const float mp = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c3;
      // (no base yet: any key raises it)
      const bool raise = mp > (m == -INFINITY ? -INFINITY : m + kRescaleLog2);
      if (__any_sync(0xffffffffu, raise) && lane == 0) bars->raise[sb][quarter][part] = J + j + 1;
      warp_arrive(&bars->s_read[quarter]);

      if (!warp_wait(smem_u32(&bars->s_read[quarter]), (J + j) & 1, a.err, abort)) { ok = false; break; }
      static_assert(kModsParts == 4, "one load");
      const int4 want = ld_shared_int4(smem_u32(bars->raise[sb][quarter]));
      const int now = J + j + 1;
      const bool raised = want.x == now || want.y == now || want.z == now || want.w == now;
      if (raised) {  // (the same for all four warps)
        float all[kModsParts];
        if (!exchange(mp, all)) { ok = false; break; }
        const float mt = fmaxf(fmaxf(all[0], all[1]), fmaxf(all[2], all[3]));
        float alpha = 1.0f;
        if (m == -INFINITY) {
          m = mt;  // nothing accumulated yet (O's row is zero or unwritten)
        } else if (mt - m > kRescaleLog2) {
          alpha = ex2_approx(m - mt);
          m = mt;
        }
        if (__any_sync(0xffffffffu, alpha != 1.0f)) {
          // A base is raised after a tile with a key (so j > 0): PV_{j-1} must be complete before O's rows are
          // scaled; PV_j is not issued until P_j below is published.
          if (!warp_wait(smem_u32(&bars->o_done[(J + j - 1) & 1]), ((J + j - 1) >> 1) & 1, a.err, abort)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < kDVP / kCW; ++cc) {
            uint32_t o[kCW];
            tmem_ld<kCW>(tmem_O + cc * kCW, o);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < kCW; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st<kCW>(tmem_O + cc * kCW, o);
          }
          tc_wait_st();
        }
        l *= alpha;
      }
      const float nb = m == -INFINITY ? 0.0f : -m;
      const float2 c32 = make_float2(c3, c3), nb2 = make_float2(nb, nb);
      uint32_t p[N / 2];
      float2 sum2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float2 t = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), c32, nb2);
        p[i] = pack_bf16x2(ex2_approx(t.x), ex2_approx(t.y));
        sum2[i & 1] = __fadd2_rn(sum2[i & 1], make_float2(bf16_lo(p[i]), bf16_hi(p[i])));
      }
      tmem_st16(tmem + lane_off + sb * kBN + part * (N / 2), p);
      l += (sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y);
      tc_wait_st();
      tc_fence_before();
      warp_arrive(&bars->p_full[sb]);
    }
    if (!ok) break;
    const Next done = cur;
    // The next item's keys are on their way while this one's output is finished.  (The producer has drawn it by now, or
    // does without waiting for any of this item's weights.)
    const bool more = fetch(n + 1, cur);
    float all[kModsParts];
    if (!exchange(l, all)) break;
    l = (all[0] + all[1]) + (all[2] + all[3]);
    // O / l as bf16, in the chunk-major 128-byte-swizzled layout of the output tensor map, into the ring slots of the
    // item's last V parts (free once the last PV has completed).  Rows past T fall outside the map and are not written.
    const int last_part = parts + ntiles * kParts - 1;  // ring sequence number
    auto oslot = [&](int k) { return (last_part - (C::OSLOTS - 1) + k) % C::NSLOT; };
    const int jl = J + ntiles - 1;
    if (!warp_wait(smem_u32(&bars->o_done[jl & 1]), (jl >> 1) & 1, a.err, abort)) break;
    tc_fence_after();
    const float inv_l = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;  // (NaN stays)
    constexpr int NCC = kDVP / kCW;
    uint32_t o[NCC][kCW];
#pragma unroll
    for (int cc = 0; cc < NCC; ++cc) tmem_ld<kCW>(tmem_O + cc * kCW, o[cc]);
    tc_wait_ld();
    uint32_t top = 0;  // largest magnitudes, as bits of bf16 pairs
#pragma unroll
    for (int cc = 0; cc < NCC; ++cc) {
      // kCW columns, half of a 64-column chunk or less: pieces (16 bytes) from p0 on
      const int col = part * kDVP + cc * kCW;
      const int ch = col / 64;
      const uint32_t row_addr = sRing + oslot(ch / C::CPS) * C::SLOTB + (ch % C::CPS) * kChunkB + r * 128;
      const int p0 = (col % 64) / 8;
#pragma unroll
      for (int i = 0; i < kCW / 8; ++i) {
        uint32_t v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k] = pack_bf16x2(__uint_as_float(o[cc][8 * i + 2 * k]) * inv_l, __uint_as_float(o[cc][8 * i + 2 * k + 1]) * inv_l);
          top = __vmaxu2(top, v[k] & 0x7fff7fffu);
        }
        const uint32_t addr = row_addr + (((p0 + i) ^ (r & 7)) * 16);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                     : "memory");
      }
    }
    // Rows with a NaN or an infinity, if only from keys that they do not see.
    // (Those whose sum is one have it from a key that they do.)
    const bool odd = max(top & 0xffffu, top >> 16) >= 0x7f80u && inv_l == inv_l && done.keys.y - done.keys.x <= kAgainKeys;
    for (unsigned todo = __ballot_sync(0xffffffffu, odd); todo != 0; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const TcItem w = tc_item<C::NDH, kMods>(a, done.it, nqt);
      const int2 keys = make_int2(__shfl_sync(0xffffffffu, done.keys.x, src), __shfl_sync(0xffffffffu, done.keys.y, src));
      const int row = quarter * 32 + src;
      const float2 v = row_again<HD, kDVP>(a, w.b, w.h, w.q0 + row, keys, __shfl_sync(0xffffffffu, done.qpos, src), done.slope,
                                           __shfl_sync(0xffffffffu, m == -INFINITY ? 0.0f : m, src),
                                           __shfl_sync(0xffffffffu, inv_l, src),
                                           w.dh * C::DV + part * kDVP);
      __syncwarp();  // (the row's first values are in place)
      if (lane * 2 < kDVP) {
        const int col = part * kDVP + lane * 2, ch = col / 64;
        const uint32_t addr = sRing + oslot(ch / C::CPS) * C::SLOTB + (ch % C::CPS) * kChunkB + row * 128 +
                              ((col % 64 / 8) ^ (row & 7)) * 16 + col % 8 * 2;
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(pack_bf16x2(v.x, v.y)) : "memory");
      }
    }
    fence_proxy_async_smem();
    // (the storing warp has seen the item before: no phase is passed over)
    if (nq > 0 && !warp_wait(smem_u32(&bars->o_taken), (nq - 1) & 1, a.err, abort)) break;
    warp_arrive(&bars->o_staged);
    J += ntiles;
    parts += ntiles * kParts;
    ++nq;
    ok = more;
  }
}

// The storing warp: the items' outputs go out from their ring slots, which are then free.
template <int HD>
__device__ __forceinline__ void store_mods(const ModsTcArgs& a, TcBars* bars, uint32_t sRing, int nqt, const CUtensorMap* tm_o) {
  using C = TcCfg<HD>;
  constexpr int kParts = C::KPARTS + C::VPARTS;
  const int lane = threadIdx.x & 31;
  volatile int* abort = &bars->abort;
  int nq = 0, parts = 0;
  for (int n = 0;; ++n) {
    const int e = n & 3;
    if (!warp_wait(smem_u32(&bars->it_full[e]), (n >> 2) & 1, a.err, abort)) break;
    const int it = *reinterpret_cast<volatile int*>(&bars->items[e]);
    const int kbeg = *reinterpret_cast<volatile int*>(&bars->kbeg[e]);
    const int kend = *reinterpret_cast<volatile int*>(&bars->kend[e]);
    warp_arrive(&bars->it_empty[e]);
    if (it < 0) break;
    TcItem w = tc_item<C::NDH, kMods>(a, it, nqt);
    tc_set_keys(w, kbeg, kend);
    if (w.ntiles == 0) continue;
    if (!warp_wait(smem_u32(&bars->o_staged), nq & 1, a.err, abort)) break;
    const int last_part = parts + w.ntiles * kParts - 1;
    auto oslot = [&](int k) { return (last_part - (C::OSLOTS - 1) + k) % C::NSLOT; };
    if (lane == 0) {
      mbar_arrive(smem_u32(&bars->o_taken));
#pragma unroll
      for (int k = 0; k < C::OSLOTS; ++k)
        tma_store_5d(tm_o, sRing + oslot(k) * C::SLOTB, 0, w.q0, w.dh * (C::DV / 64) + k * C::CPS, w.h, w.b);
      bulk_commit_group();
      bulk_wait_read_all();  // the slots must not be refilled before the stores have read them
#pragma unroll
      for (int k = 0; k < C::OSLOTS; ++k) mbar_arrive(smem_u32(&bars->empty[oslot(k)]));
    }
    __syncwarp();
    parts += w.ntiles * kParts;
    ++nq;
  }
}

// (CAP and BIAS: with MODS, whether scores are capped and biased)
template <int HD, int MODE, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads<MODE>, 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                      const __grid_constant__ TcArgsOf<MODE> a) {
  using C = TcCfg<HD>;
  constexpr bool BIDIR = MODE == kBidir;
  constexpr bool MODS = MODE == kMods;
  // 128-byte-swizzled tiles need 1024-byte alignment; the declaration asks
  // for it, and a block that does not get it reports and does nothing.
  extern __shared__ __align__(1024) uint8_t smem[];
  // The last CTA to finish clears the launch's work-item counters for the
  // next launch that uses them (every CTA has drawn its last item by then).
  auto release_counters = [&]() {
    if (threadIdx.x == 0) {
      __threadfence();
      if (atomicAdd(a.item_ctr + 1, 1u) == gridDim.x - 1) {
        __threadfence();
        atomicExch(a.item_ctr, 0u);
        atomicExch(a.item_ctr + 1, 0u);
      }
    }
  };
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicExch(a.err, kErrSmemAlign);
    release_counters();
    return;
  }
  TcBars* bars = reinterpret_cast<TcBars*>(smem + C::BAR_OFF);
  const uint32_t sQ = smem_u32(smem + C::Q_OFF);
  const uint32_t sRing = smem_u32(smem + C::RING_OFF);
  volatile int* abort = &bars->abort;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if constexpr (!MODS) pdl_wait();  // (MODS: once the barriers are set up)
  pdl_trigger();

  const int nqt = (a.T + kBM - 1) / kBM;
  const int nitems = nqt * a.H * a.B * C::NDH;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars->q_full), 1);
    mbar_init(smem_u32(&bars->q_free), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->s_full[i]), 1);
      mbar_init(smem_u32(&bars->p_full[i]), MODS ? kSoftWarps<MODE> : 256);
      mbar_init(smem_u32(&bars->o_done[i]), 1);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    for (int qq = 0; qq < 4; ++qq) mbar_init(smem_u32(&bars->sum_full[qq]), 64);
    for (int qq = 0; qq < 4; ++qq) mbar_init(smem_u32(&bars->s_read[qq]), MODS ? kModsParts : 64);
    if constexpr (MODS) {
      // (warps are counted, whose lane 0 arrives for them)
      for (int qq = 0; qq < 4; ++qq) {
        mbar_init(smem_u32(&bars->x_full[qq]), kModsParts);
        mbar_init(smem_u32(&bars->x_free[qq]), kModsParts);
      }
      mbar_init(smem_u32(&bars->o_staged), kSoftWarps<MODE>);
      mbar_init(smem_u32(&bars->o_taken), 1);
      for (int i = 0; i < 2 * 4 * kModsParts; ++i) (&bars->raise[0][0][0])[i] = 0;
    }
    for (int i = 0; i < C::NSLOT; ++i) mbar_init(smem_u32(&bars->full[i]), 1);
    for (int i = 0; i < C::NSLOT; ++i) mbar_init(smem_u32(&bars->empty[i]), 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&bars->it_full[i]), 1);
      mbar_init(smem_u32(&bars->it_empty[i]), MODS ? 2 + kSoftWarps<MODE> : 2);  // its readers
    }
    bars->abort = 0;
    fence_mbar_init();
  }
  // (after the wait: TMEM taken while the launch before has yet to take its own could leave both waiting)
  if constexpr (MODS) pdl_wait();
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const uint32_t tmem_O = tmem + 256;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // The warp runs the loop converged; one elected lane draws the work items
    // and issues every copy.  The ring runs on across work items: the next
    // item's Q is loaded once the last QK MMA of the current one has read the
    // old Q, and its first K parts go into whatever slots are free while the
    // current item finishes.
    {
      if (elect_one()) {
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
      }
      __syncwarp();
      const uint32_t qb = smem_u32(&bars->q_full);
      bool ok = true;
      int seq = 0;
      int slot = 0;        // ring slot of the next part
      uint32_t phase = 0;  // parity of that slot's current use
      int nq = 0;          // items whose Q has been requested
      auto advance = [&]() {
        ++seq;
        if (++slot == C::NSLOT) {
          slot = 0;
          phase ^= 1u;
        }
      };
      for (int n = 0; ok; ++n) {
        // next work item into queue entry n % 4 (once both readers are done with its last use)
        const int e = n & 3;
        if (n >= 4 && !warp_wait(smem_u32(&bars->it_empty[e]), ((n >> 2) - 1) & 1, a.err, abort)) break;
        unsigned got = blockIdx.x;
        if (!MODS || n > 0) {  // (MODS: a CTA's first item is its own, the counter gives out the others)
          if (lane == 0) got = atomicAdd(a.item_ctr, 1u) + (MODS ? gridDim.x : 0u);
          got = __shfl_sync(0xffffffffu, got, 0);
        }
        const int it = got < static_cast<unsigned>(nitems) ? static_cast<int>(got) : -1;
        TcItem w;
        if constexpr (MODS) {
          // the keys that some row of the tile sees
          int lo = 0x7fffffff, hi = 0;
          if (it >= 0) {
            w = tc_item<C::NDH, MODE>(a, it, nqt);
#pragma unroll
            for (int i = 0; i < kBM / 32; ++i) {
              const int2 keys = tc_row_keys(a, w, lane + 32 * i);
              if (keys.x < keys.y) {
                lo = min(lo, keys.x);
                hi = max(hi, keys.y);
              }
            }
            lo = __reduce_min_sync(0xffffffffu, lo);
            hi = __reduce_max_sync(0xffffffffu, hi);
            if (hi == 0) lo = 0;
            tc_set_keys(w, lo, hi);
          }
          if (lane == 0) {
            *reinterpret_cast<volatile int*>(&bars->kbeg[e]) = lo;
            *reinterpret_cast<volatile int*>(&bars->kend[e]) = hi;
          }
        }
        if (lane == 0) {
          *reinterpret_cast<volatile int*>(&bars->items[e]) = it;
          mbar_arrive(smem_u32(&bars->it_full[e]));
        }
        __syncwarp();
        if (it < 0) break;
        if constexpr (!MODS) w = tc_item<C::NDH, MODE>(a, it, nqt);
        if (w.ntiles == 0) continue;
        if (nq > 0 && !warp_wait(smem_u32(&bars->q_free), (nq - 1) & 1, a.err, abort)) break;
        // Q tile: 128 rows x QCH chunks in one request (two for head_dim 512)
        constexpr int QREQ = C::QCH > 4 ? 2 : 1;
        if (elect_one()) {
          mbar_arrive_expect_tx(qb, C::QCH * kChunkB);
#pragma unroll
          for (int r = 0; r < QREQ; ++r)
            tma_load_5d(sQ + r * (C::QCH / QREQ) * kChunkB, &tm_q, 0, w.q0, r * (C::QCH / QREQ), w.h, w.b, qb);
        }
        __syncwarp();
        ++nq;
        // Cache row of a key tile's first position: on a ring of max_len
        // rows (a multiple of the 128-key tile, so no tile wraps) the
        // position modulo max_len.
        auto tile_row = [&](int kt) { return a.ring ? (kt * kBN) % a.max_len : kt * kBN; };
        auto load_k = [&](int kt) {
          const int kr = tile_row(kt);
          for (int p2 = 0; p2 < C::KPARTS && ok; ++p2) {
            if (!warp_wait(smem_u32(&bars->empty[slot]), phase ^ 1u, a.err, abort)) { ok = false; break; }
            const uint32_t fb = smem_u32(&bars->full[slot]);
            if (elect_one()) {
              mbar_arrive_expect_tx(fb, C::KPB);
              tma_load_5d(sRing + slot * C::SLOTB, &tm_k, 0, kr, p2 * C::CPP, w.kvh, w.b, fb);
            }
            __syncwarp();
            advance();
          }
        };
        auto load_v = [&](int kt) {
          const int kr = tile_row(kt);
          for (int p2 = 0; p2 < C::VPARTS && ok; ++p2) {
            if (!warp_wait(smem_u32(&bars->empty[slot]), phase ^ 1u, a.err, abort)) { ok = false; break; }
            const uint32_t fb = smem_u32(&bars->full[slot]);
            if (elect_one()) {
              mbar_arrive_expect_tx(fb, C::VPB);
              tma_load_5d(sRing + slot * C::SLOTB, &tm_v, 0, kr + p2 * C::VKP, w.dh * (C::DV / 64), w.kvh, w.b,
                          fb);
            }
            __syncwarp();
            advance();
          }
        };
        auto tile = [&](int j) { return MODS ? w.kt_begin + w.ntiles - 1 - j : w.kt_begin + j; };
        load_k(tile(0));
        for (int j = 0; j < w.ntiles && ok; ++j) {
          if (j + 1 < w.ntiles) load_k(tile(j + 1));
          load_v(tile(j));
        }
      }
      // Copies still in flight must land before the CTA may exit.
      if (nq > 0) warp_wait(qb, (nq - 1) & 1, nullptr);
      for (int s2 = max(0, seq - C::NSLOT); s2 < seq; ++s2)
        warp_wait(smem_u32(&bars->full[s2 % C::NSLOT]), (s2 / C::NSLOT) & 1, nullptr);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the issue loop converged (waits included) and one
    // elected lane issues each tcgen05.mma and commit: the loop's descriptor
    // and ring arithmetic stays warp-uniform, and issue keeps ahead of the
    // tensor pipe (run by one lane inside a lane test, the loop issued each
    // MMA slower than the pipe executes it).  Tile parities run on across
    // items (J counts every tile of the CTA).
    {
      constexpr uint32_t idesc_qk = idesc_bf16_f32(kBM, kBN, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(kBM, C::DV, 0, 1);
      bool ok = true;
      // Descriptors are built once; a slot, a 64-dim chunk or a 16-element
      // K step only moves the start address (16-byte units in the low bits,
      // which stay below 2^14 for any shared-memory address).  Building them
      // per instruction costs the issue loop more cycles than the MMA.
      const uint32_t lead = elect_one();  // (asked once: an elect per MMA costs the issue loop 1-3 %)
      const uint64_t dq0 = smem_desc_sw128(sQ, 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(sRing, 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(sRing, C::VKP * 128, 1024);
      // Ring state, advanced incrementally: the issue loop's own instruction
      // latency sits between MMAs of 64 cycles, so there is no division,
      // modulo or multiply on this path.
      int slot = 0;        // ring slot of the next part
      uint32_t phase = 0;  // parity of that slot's current use
      uint32_t soff = 0;   // slot * SLOTB in descriptor units (16 bytes)
      const uint32_t full0 = smem_u32(&bars->full[0]);
      const uint32_t empty0 = smem_u32(&bars->empty[0]);
      auto advance = [&]() {
        soff += C::SLOTB >> 4;
        if (++slot == C::NSLOT) {
          slot = 0;
          phase ^= 1u;
          soff = 0;
        }
      };
      auto release = [&]() {
        tc_commit_elect(empty0 + slot * 8);
        advance();
      };
      int J = 0;   // tiles of earlier items
      int nq = 0;  // items started
      for (int n = 0; ok; ++n) {
        const int e = n & 3;
        if (!warp_wait(smem_u32(&bars->it_full[e]), (n >> 2) & 1, a.err, abort)) break;
        const int it = *reinterpret_cast<volatile int*>(&bars->items[e]);
        [[maybe_unused]] int kbeg = 0, kend = 0;
        if constexpr (MODS) {
          kbeg = *reinterpret_cast<volatile int*>(&bars->kbeg[e]);
          kend = *reinterpret_cast<volatile int*>(&bars->kend[e]);
          __syncwarp();  // (every lane has read the entry before it is given back)
        }
        if (lane == 0) mbar_arrive(smem_u32(&bars->it_empty[e]));
        __syncwarp();
        if (it < 0) break;
        TcItem w = tc_item<C::NDH, MODE>(a, it, nqt);
        if constexpr (MODS) tc_set_keys(w, kbeg, kend);
        if (w.ntiles == 0) continue;
        if (!warp_wait(smem_u32(&bars->q_full), nq & 1, a.err, abort)) break;
        ++nq;
        tc_fence_after();
        auto mma_qk = [&](int j) {
          const int sb = (J + j) & 1;
          const uint32_t dS = tmem + sb * kBN;
          uint64_t ad = dq0;
#pragma unroll 1
          for (int p2 = 0; p2 < C::KPARTS; ++p2) {
            if (!warp_wait(full0 + slot * 8, phase, a.err, abort)) { ok = false; return; }
            tc_fence_after();
            uint64_t bd = dk0 + soff;
#pragma unroll
            for (int c = 0; c < C::CPP; ++c) {
              tc_mma_ss_lead(lead, dS, ad, bd, idesc_qk, (p2 > 0 || c > 0) ? 1u : 0u);
              tc_mma_ss_lead(lead, dS, ad + 2, bd + 2, idesc_qk, 1u);
              tc_mma_ss_lead(lead, dS, ad + 4, bd + 4, idesc_qk, 1u);
              tc_mma_ss_lead(lead, dS, ad + 6, bd + 6, idesc_qk, 1u);
              ad += kChunkB >> 4;
              bd += kChunkB >> 4;
            }
            release();
          }
          tc_commit_elect(smem_u32(&bars->s_full[sb]));
          // after the item's last QK, the Q area may take the next item's Q
          if (j == w.ntiles - 1) tc_commit_elect(smem_u32(&bars->q_free));
        };
        auto mma_pv = [&](int j) {
          const int sb = (J + j) & 1;
          if (!warp_wait(smem_u32(&bars->p_full[sb]), ((J + j) >> 1) & 1, a.err, abort)) { ok = false; return; }
          tc_fence_after();
          const int kt = MODS ? w.kt_begin + w.ntiles - 1 - j : w.kt_begin + j;
          uint32_t ta = tmem + sb * kBN;  // P_j: 128 keys as 64 packed columns
          const bool last = j == w.ntiles - 1;
#pragma unroll 1
          for (int p2 = 0; p2 < C::VPARTS; ++p2) {
            if (!warp_wait(full0 + slot * 8, phase, a.err, abort)) { ok = false; return; }
            // Rows of keys past the cache's filled length may hold anything
            // (even NaN, and 0 * NaN = NaN); zero them before they meet P
            // (only in the part holding the end of the keys).
            const int key0 = kt * kBN + p2 * C::VKP;
            // A 64-column chunk of a part is 128 bytes per key, key after key (the swizzle stays within a key's).
            auto zero_keys = [&](int first, int count) {
              uint8_t* from = smem + C::RING_OFF + slot * C::SLOTB + first * 128;
#pragma unroll
              for (int dc = 0; dc < C::DV / 64; ++dc)
                for (int i = lane * 16; i < count * 128; i += 512)
                  *reinterpret_cast<uint4*>(from + dc * C::VKP * 128 + i) = make_uint4(0, 0, 0, 0);
              fence_proxy_async_smem();
              __syncwarp();
            };
            const int nvalid = keys_before(w.Lk, key0, C::VKP);
            if (nvalid < C::VKP) zero_keys(nvalid, C::VKP - nvalid);
            if constexpr (MODS) {
              // and so may those before the first key that a row sees
              if (key0 < w.kbeg) zero_keys(0, min(C::VKP, w.kbeg - key0));
            }
            tc_fence_after();
            const uint64_t bd = dv0 + soff;
#pragma unroll
            for (int kk = 0; kk < C::VKP / 16; ++kk)
              tc_mma_ts_lead(lead, tmem_O, ta + kk * 8, bd + static_cast<uint64_t>(kk * 128), idesc_pv,
                        (j > 0 || p2 > 0 || kk > 0) ? 1u : 0u);
            ta += C::VKP / 2;
            // The item's last OSLOTS V parts stay held: the epilogue stages
            // O there and frees them after its store has read them.
            if (last && p2 >= C::VPARTS - C::OSLOTS)
              advance();
            else
              release();
          }
          tc_commit_elect(smem_u32(&bars->o_done[sb]));
        };
        mma_qk(0);
        for (int j = 0; j < w.ntiles && ok; ++j) {
          if (j + 1 < w.ntiles) mma_qk(j + 1);
          if (ok) mma_pv(j);
        }
        J += w.ntiles;
      }
      // Every MMA issued so far completes before TMEM is released.
      tc_commit_elect(smem_u32(&bars->drain));
      warp_wait(smem_u32(&bars->drain), 0, nullptr);
    }
    __syncwarp();
  } else if constexpr (MODS) {
    if (warp < 2 + kSoftWarps<MODE>)
      softmax_mods<HD, CAP, BIAS>(a, bars, tmem, sRing, nqt);
    else
      store_mods<HD>(a, bars, sRing, nqt, &tm_o);
  } else {
    // ------------------------------------------------------------ softmax
    const int quarter = warp & 3;  // TMEM lane quarter this warp may access
    const int half = (warp - 2) >> 2;  // which 64 of the 128 score columns
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const float c2 = a.scale_log2;  // > 0 (checked on the host)
    constexpr int kHB = kBN / 2;    // score columns per thread
    constexpr int kDVH = C::DV / 2; // O columns per thread
    constexpr int kParts = C::KPARTS + C::VPARTS;  // ring parts per key tile
    int J = 0;      // tiles of earlier items
    int nq = 0;     // items done
    int parts = 0;  // ring parts of earlier items
    for (int n = 0;; ++n) {
      const int e = n & 3;
      const int it = warp_wait(smem_u32(&bars->it_full[e]), (n >> 2) & 1, a.err, abort)
                         ? *reinterpret_cast<volatile int*>(&bars->items[e])
                         : -1;
      if (it < 0) {
        // no item left (or a wait gave up): every softmax thread leaves here
        // or at the end of an item, together
        softmax_sync_any(1);
        break;
      }
      const TcItem w = tc_item<C::NDH, MODE>(a, it, nqt);
      const int ntiles = w.ntiles;
      if (ntiles == 0) {
        // No visible key (only reachable with out-of-contract positions).
        if (r < w.valid_rows) {
          __nv_bfloat16* dst =
              static_cast<__nv_bfloat16*>(a.out) +
              (((static_cast<size_t>(w.b) * a.T + w.q0 + r) * a.H + w.h) * HD + w.dh * C::DV + half * kDVH);
          for (int i = 0; i < kDVH / 8; ++i) reinterpret_cast<uint4*>(dst)[i] = make_uint4(0, 0, 0, 0);
        }
        const bool stop0 = softmax_sync_any(*abort);
        if (warp == 2 && lane == 0 && !stop0) mbar_arrive(smem_u32(&bars->it_empty[e]));
        __syncwarp();
        if (stop0) break;
        continue;
      }
      const int qpos = w.qpos_first + r;
      const bool row_valid = r < w.valid_rows;
      float m = -INFINITY;  // exponent base in log2 units: a stale running maximum
      float l = 0.0f;       // this half's share of the row sum
      bool ok = true;
      for (int j = 0; j < ntiles; ++j) {
        const int sb = (J + j) & 1;
        if (!warp_wait(smem_u32(&bars->s_full[sb]), ((J + j) >> 1) & 1, a.err, abort)) { ok = false; break; }
        tc_fence_after();
        float s[kHB];
        float mt;
        {
          // the whole row: both threads of a row take the same maximum
          uint32_t r0[32], r1[32], o0[32], o1[32];
          const uint32_t tS = tmem + lane_off + sb * kBN;
          tmem_ld32(tS + half * kHB, r0);
          tmem_ld32(tS + half * kHB + 32, r1);
          tmem_ld32(tS + (1 - half) * kHB, o0);
          tmem_ld32(tS + (1 - half) * kHB + 32, o1);
          tc_wait_ld();
          // P_j goes over S_j, partly over the other warp's half of the row,
          // which that warp reads too: tell it this warp's reads are done.
          mbar_arrive(smem_u32(&bars->s_read[quarter]));
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            s[i] = __uint_as_float(r0[i]);
            s[32 + i] = __uint_as_float(r1[i]);
          }
          const int kr = (w.kt_begin + j) * kBN;
          const bool row_vis =
              BIDIR ? row_valid && (kr + kBN <= w.Lk) &&
                          (!a.sliding || (qpos - kr <= a.window && kr + kBN - 1 - qpos <= a.window))
                    : row_valid && (kr + kBN - 1 <= qpos) && (kr + kBN <= w.Lk) &&
                          (!a.sliding || qpos - kr < a.window);
          const int k0 = kr + half * kHB;
          const int k1 = kr + (1 - half) * kHB;
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if (row_vis) {
#pragma unroll
            for (int n = 0; n < 32; ++n) {
              mx[n & 3] = fmaxf(mx[n & 3], fmaxf(s[n], s[32 + n]));
              mx[(n + 2) & 3] = fmaxf(mx[(n + 2) & 3], fmaxf(__uint_as_float(o0[n]), __uint_as_float(o1[n])));
            }
          } else {
            // The row's visible keys are one interval [vlo, vhi): causal end,
            // the cache's filled length and (sliding) the window start; in
            // the encoder form the window's two ends and the sequence end.
            const int vlo = a.sliding ? max(0, qpos - a.window + (BIDIR ? 0 : 1)) : 0;
            const int vhi = !row_valid ? 0
                            : BIDIR    ? (a.sliding ? min(qpos + a.window + 1, w.Lk) : w.Lk)
                                       : min(qpos + 1, w.Lk);
            const unsigned span = static_cast<unsigned>(max(0, vhi - vlo));
            const int lo0 = vlo - k0, lo1 = vlo - k1;
#pragma unroll
            for (int n = 0; n < kHB; ++n) {
              if (static_cast<unsigned>(n - lo0) >= span) s[n] = -INFINITY;
              mx[n & 3] = fmaxf(mx[n & 3], s[n]);
            }
#pragma unroll
            for (int n = 0; n < 32; ++n) {
              const float v0 = static_cast<unsigned>(n - lo1) < span ? __uint_as_float(o0[n]) : -INFINITY;
              const float v1 = static_cast<unsigned>(n + 32 - lo1) < span ? __uint_as_float(o1[n]) : -INFINITY;
              mx[n & 3] = fmaxf(mx[n & 3], fmaxf(v0, v1));
            }
          }
          mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
        }
        float alpha = 1.0f;
        bool rescale = false;
        float m_use = m;
        if (m == -INFINITY) {
          m_use = mt;  // nothing accumulated yet (O row is zero or unwritten)
        } else if (mt - m > kRescaleLog2) {
          m_use = mt;
          alpha = ex2_approx(m - mt);
          rescale = true;
        }
        if (__any_sync(0xffffffffu, rescale)) {
          // A row of this warp raises its base (only after a tile with a
          // visible key, so j > 0): PV_{j-1} must be complete before the O
          // rows are scaled; PV_j is not issued until P_j below is published.
          if (!warp_wait(smem_u32(&bars->o_done[(J + j - 1) & 1]), ((J + j - 1) >> 1) & 1, a.err, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float f = rescale ? alpha : 1.0f;
#pragma unroll 1
          for (int cc = 0; cc < kDVH / 32; ++cc) {
            uint32_t rr[32];
            const uint32_t tO = tmem_O + lane_off + half * kDVH + cc * 32;
            tmem_ld32(tO, rr);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) rr[i] = __float_as_uint(__uint_as_float(rr[i]) * f);
            tmem_st32(tO, rr);
          }
          tc_wait_st();
        }
        const float nb = (m_use == -INFINITY) ? 0.0f : -m_use;
        uint32_t p[32];
        float sa[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint32_t pw = pack_bf16x2(ex2_approx(fmaf(s[2 * i], c2, nb)), ex2_approx(fmaf(s[2 * i + 1], c2, nb)));
          p[i] = pw;
          sa[(2 * i) & 3] += bf16_lo(pw);
          sa[(2 * i + 1) & 3] += bf16_hi(pw);
        }
        if (!warp_wait(smem_u32(&bars->s_read[quarter]), (J + j) & 1, a.err, abort)) {
          ok = false;
          break;
        }
        tmem_st32(tmem + lane_off + sb * kBN + half * (kHB / 2), p);
        l = l * alpha + ((sa[0] + sa[1]) + (sa[2] + sa[3]));
        m = m_use;
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&bars->p_full[sb]));
      }
      if (ok) {
        // the full row sum: both halves' shares
        bars->red[half][r] = l;
        mbar_arrive(smem_u32(&bars->sum_full[quarter]));
        ok = warp_wait(smem_u32(&bars->sum_full[quarter]), nq & 1, a.err, abort);
        l = bars->red[0][r] + bars->red[1][r];
      }
      // Epilogue: O / l as bf16, in the chunk-major 128-byte-swizzled layout of
      // the output tensor map, into the ring slots of the item's last V parts
      // (free once the last PV has completed), then TMA stores of the tile.
      // Rows past T fall outside the map and are not written.
      const int last_part = parts + ntiles * kParts - 1;  // ring sequence number
      auto oslot = [&](int k) { return (last_part - (C::OSLOTS - 1) + k) % C::NSLOT; };
      if (ok) {
        const int jl = J + ntiles - 1;
        if (warp_wait(smem_u32(&bars->o_done[jl & 1]), (jl >> 1) & 1, a.err, abort)) {
          tc_fence_after();
          const float inv_l = l > 0.0f ? 1.0f / l : 0.0f;
          constexpr int NCC = kDVH / 32;
          uint32_t rr[NCC][32];
#pragma unroll
          for (int cc = 0; cc < NCC; ++cc) tmem_ld32(tmem_O + lane_off + half * kDVH + cc * 32, rr[cc]);
          tc_wait_ld();
#pragma unroll
          for (int cc = 0; cc < NCC; ++cc) {
            // 32 columns = half a 64-column chunk: pieces (16 bytes) p0 .. p0 + 3
            const int col = half * kDVH + cc * 32;
            const int ch = col / 64;
            const uint32_t row_addr = sRing + oslot(ch / C::CPS) * C::SLOTB + (ch % C::CPS) * kChunkB + r * 128;
            const int p0 = (col % 64) / 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t x = pack_bf16x2(__uint_as_float(rr[cc][8 * i + 0]) * inv_l, __uint_as_float(rr[cc][8 * i + 1]) * inv_l);
              const uint32_t y = pack_bf16x2(__uint_as_float(rr[cc][8 * i + 2]) * inv_l, __uint_as_float(rr[cc][8 * i + 3]) * inv_l);
              const uint32_t z = pack_bf16x2(__uint_as_float(rr[cc][8 * i + 4]) * inv_l, __uint_as_float(rr[cc][8 * i + 5]) * inv_l);
              const uint32_t q = pack_bf16x2(__uint_as_float(rr[cc][8 * i + 6]) * inv_l, __uint_as_float(rr[cc][8 * i + 7]) * inv_l);
              const uint32_t addr = row_addr + (((p0 + i) ^ (r & 7)) * 16);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(q)
                           : "memory");
            }
          }
          fence_proxy_async_smem();
        } else {
          ok = false;
        }
      }
      // All 256 softmax threads meet here on every path, and all leave the
      // item loop together if any wait anywhere gave up.
      const bool stop = softmax_sync_any(!ok || *abort);
      if (warp == 2 && lane == 0 && !stop) {
#pragma unroll
        for (int k = 0; k < C::OSLOTS; ++k)
          tma_store_5d(&tm_o, sRing + oslot(k) * C::SLOTB, 0, w.q0, w.dh * (C::DV / 64) + k * C::CPS, w.h, w.b);
        bulk_commit_group();
        bulk_wait_read_all();  // the slots must not be refilled before the stores have read them
#pragma unroll
        for (int k = 0; k < C::OSLOTS; ++k) mbar_arrive(smem_u32(&bars->empty[oslot(k)]));
      }
      if (warp == 2 && lane == 0 && !stop) mbar_arrive(smem_u32(&bars->it_empty[e]));
      __syncwarp();
      if (stop) break;
      J += ntiles;
      parts += ntiles * kParts;
      ++nq;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  release_counters();
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

// bf16 5-D tensor map, dims innermost first, 128-byte swizzle, zero fill out
// of bounds.  Dim 0 is 64 consecutive elements (one 128-byte row), dim 1 the
// rows (tokens or keys), dim 2 the 64-element chunks of a head, so a box of
// (64, rows, chunks) lands in shared memory as chunk-major 128-byte rows:
// the layout the MMA descriptors read.
bool make_map(CUtensorMap* m, const void* base, const cuuint64_t dims[5], const cuuint64_t strides_bytes[4],
              const cuuint32_t box[5]) {
  EncodeTiledFn fn = get_encode_fn();
  if (fn == nullptr) return false;
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides_bytes, box,
                        estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

template <int HD, int MODE, bool CAP = false, bool BIAS = false>
cudaError_t launch_hd(const TcArgsOf<MODE>& a, cudaStream_t s) {
  using C = TcCfg<HD>;
  const cudaError_t e = set_smem_limit_once<prefill_tc_kernel<HD, MODE, CAP, BIAS>>(C::SMEM_B);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv, mo;
  const cuuint64_t row_b = static_cast<cuuint64_t>(HD) * 2;
  constexpr cuuint32_t kQBoxChunks = C::QCH > 4 ? C::QCH / 2 : C::QCH;
  {
    // q [B][T][H][hd]: (element, token, chunk, head, sequence)
    const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(a.T), static_cast<cuuint64_t>(C::QCH),
                                static_cast<cuuint64_t>(a.H), static_cast<cuuint64_t>(a.B)};
    const cuuint64_t str[4] = {row_b * a.H, 128, row_b, row_b * a.H * a.T};
    const cuuint32_t box[5] = {64, kBM, kQBoxChunks, 1, 1};
    if (!make_map(&mq, a.q, dims, str, box)) return cudaErrorInvalidValue;
  }
  {
    // cache [B][Hkv][max_len][hd]: (element, key, chunk, kv head, sequence)
    const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(a.max_len), static_cast<cuuint64_t>(C::QCH),
                                static_cast<cuuint64_t>(a.Hkv), static_cast<cuuint64_t>(a.B)};
    const cuuint64_t str[4] = {row_b, 128, row_b * a.max_len, row_b * a.max_len * a.Hkv};
    const cuuint32_t boxk[5] = {64, kBN, C::CPP, 1, 1};
    const cuuint32_t boxv[5] = {64, C::VKP, C::DV / 64, 1, 1};
    if (!make_map(&mk, a.ck, dims, str, boxk)) return cudaErrorInvalidValue;
    if (!make_map(&mv, a.cv, dims, str, boxv)) return cudaErrorInvalidValue;
  }
  {
    // out [B][T][H][hd], written DV columns (DV / 64 chunks) at a time
    const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(a.T), static_cast<cuuint64_t>(C::QCH),
                                static_cast<cuuint64_t>(a.H), static_cast<cuuint64_t>(a.B)};
    const cuuint64_t str[4] = {row_b * a.H, 128, row_b, row_b * a.H * a.T};
    const cuuint32_t box[5] = {64, kBM, C::CPS, 1, 1};
    if (!make_map(&mo, a.out, dims, str, box)) return cudaErrorInvalidValue;
  }
  // One persistent CTA per SM (shared memory and TMEM allow no more), each
  // drawing work items from the launch's counter pair until none is left.
  const int nqt = (a.T + kBM - 1) / kBM;
  const long long nitems = static_cast<long long>(nqt) * a.H * a.B * C::NDH;
  if (nitems > 0x7fffffffLL) return cudaErrorInvalidValue;
  const long long nblk = nitems < sm_count() ? nitems : sm_count();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(nblk));
  cfg.blockDim = dim3(kThreads<MODE>);
  cfg.dynamicSmemBytes = C::SMEM_B;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_tc_kernel<HD, MODE, CAP, BIAS>, mq, mk, mv, mo, a);
}

}  // namespace
}  // namespace g4
