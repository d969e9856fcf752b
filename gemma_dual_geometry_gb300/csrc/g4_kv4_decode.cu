// Decode attention over the paged 4-bit KV cache: one query per sequence,
// split over the key range (split-KV), HBM-bound.
//
// out_h = sum_j p_j v_j / sum_j p_j,  p_j = 2^(c (q_h . k_j) - m),  over the keys
// [max(0, L - window), L) (all L on full layers), c = attn_scale log2(e).
//
// All G <= 8 query heads of a kv head are served together, so a record of the
// cache (16 positions, 18 head_dim bytes) is read once.  At 4.5 bits per
// element an SM's share of HBM is ~42 elements per clock, each of which meets
// 8 (padded) heads twice: more multiply-adds than the CUDA cores have, so both
// products run on mma.sync m16n8k16 (fp16 operands, float32 sums), whose
// 16 x 16 operand is a record's scale block and whose 8 columns are the heads:
//   S^T[16 positions][8 heads] += s . (K[16 x 16] Q^T)    per 16 elements: the
//     product of the bare codes, scaled by the block's scale in float32;
//   O^T[16 elements][8 heads]  += V^T[16 x 16] (P s)^T    per 16 elements: the
//     scale of V goes into the probabilities (rounded to fp16).
// (Eight rows fill a sixteenth of a tcgen05 tile, and the operands would
// have to be widened into shared memory first.)  The cache's byte order gives
// each lane its fragments in 16-byte loads, free of bank conflicts; codes widen
// two at a time with one conversion.
//
// Work.  The records of all (sequence, kv head) units, laid end to end, are
// dealt out in equal contiguous shares to as many CTAs as are resident, so
// ragged lengths leave no SM idle.  Where that makes no share much longer, they are
// cut anew at every unit instead, so that no CTA pays for the start of a second
// one.  A unit inside one share is written directly;
// the CTAs of a unit that spans shares leave partials in the workspace and the one
// that takes the last ticket merges them.
//
// A CTA takes STEP records per step.  A fifth warp issues the copies; each of the
// other four scores its share of
// them and forms their probabilities; after a CTA barrier each warp adds all the
// step's P V for its own slice of head_dim, so O takes few registers and needs no
// merge between warps (at head_dim 64 and 128, whose 64-element pieces are
// fewer than the warps, 4 or 2 warps hold a piece and split the records).  K and V
// parts of a record are separate bulk copies in the order K_0 V_0 K_1 V_1 ...
// through a ring of SLOTS buffers: a step's K buffer is free at its barrier, its V
// buffer at the next step's.  The copies run on across the units of a share.
//
// With at most 4 heads the other 4 columns serve a second scale block, so that
// scales are handled once for two blocks.  Scores: the contraction takes 8
// elements of block 2j and 8 of block 2j + 1, q being zero for the other
// block's elements in columns 0-3 and 4-7; two products give the two blocks'
// sums side by side.  P V: the operand's rows are 8 elements of block 2j and 8 of
// block 2j + 1, columns 0-3 carry P times the scales of 2j and 4-7 of 2j + 1.
//
// The online softmax keeps a reference m per head, common to the CTA, that
// only moves (rescaling O) when a score exceeds it by 2^kSlack, so most steps
// need no reduction over positions.  Probabilities are formed as
// 2^(s - m + kShift): fp16's 11 bits then reach down to 2^-18 of the reference.
//
// Measured (device time, calls back to back; copy rate: 6.78 TB/s):
//   head_dim 512, 8 heads, 2 kv heads, 4 sequences of 131072 keys (604 MB) 110.7 us,
//     5.5 TB/s, 0.80 of a copy; every product left out: 101 us, so the copies (3
//     CTAs of 3 x 18 KB per SM, issued again at the CTA's barrier) bound it;
//   the same, 64 sequences of 1024 to 8192 keys (340 MB) 70.5 us, 0.71 of a copy:
//     the start (lengths, block ids, first copies) and the merges take 8 us;
//   head_dim 256, window 512, 64 sequences (19 MB) 13.2 us; head_dim 128, one of 333
//     keys 6.6 us: latency of that chain (the bytes take 2.9 and 0.01 us).
//   head_dim 256, 64 sequences of 1024 to 8192 keys, 8 heads per kv head 52.6 us, 4
//     heads 46.1 us.
#include <math.h>

#include "g4_device.cuh"
#include "g4_kv4_internal.h"
#include "g4_kv4.cuh"

namespace g4 {
namespace {

constexpr int kHeads = 8;  // columns of the tensor-core product
constexpr float kSlack = 3.0f;  // (0, a reference that follows every maximum: 0.6 % slower at 4 x 131072 keys)
constexpr float kShift = 4.0f;  // (2^(kSlack + kShift) times the largest scale, 448, stays within fp16)
constexpr float kNoKey = -3e38f;  // reference of a state that has seen no key (finite: no inf - inf)
// Partials merged at once.  6: 113.6 us at 4 x 131072 keys against 110.6 (more
// levels); 16: 113.8, and 15.4 against 13.2 at 64 windows (more loads than registers).
constexpr int kFan = 8;
// Shares are cut at units where that makes the longest at most so many steps longer.
// Never: 15.6 us against 13.3 at 64 windows of 512 (head_dim 256), 30.2 against 26.4
// at 256 of them, 23.4 against 15.8 at 16 sequences of 100 to 2000 keys (head_dim 512),
// 48.8 against 45.6 at 32 of 1000 to 8000.  2 to 6 steps: the same; 8: 82 against 70.5
// at 64 sequences of 1024 to 8192 keys.
constexpr int kCutSteps = 4;

// Shape of the kernel at one head_dim (also used by the plan).
template <int HD>
struct Kv4Cfg {
  static constexpr int W = 4;                                   // warps that compute
  static constexpr int NT = (W + 1) * 32;                       // and one that copies
  static constexpr int NP = HD / 64;                            // pieces of a row
  static constexpr int RW = HD >= 256 ? 1 : 256 / HD;           // records a warp scores per step
  static constexpr int STEP = W * RW;                           // records per step
  static constexpr int PW = NP >= W ? NP / W : 1;               // pieces of O per warp
  static constexpr int KS = NP >= W ? 1 : W / NP;               // warps that share a piece
  // CTAs per SM, and the buffers that this leaves room for.  At 512: 2 CTAs of 5
  // buffers the same within 1 %, 3 of 2 10 % slower.  At 256 (64 windows): 3 CTAs of
  // 6 buffers 14.1 us, 5 of 4 14.0, 4 of 4 13.2.
  static constexpr int MINB = HD >= 512 ? 3 : 4;
  static constexpr int SLOTS = HD >= 512 ? 3 : 4;
  static constexpr int HALF_B = 9 * HD;                         // K (or V) part of a record
  static constexpr int SLOT_B = STEP * HALF_B;
  static constexpr int Q_OFF = SLOTS * SLOT_B;                  // q fragments, fp16 (8 columns)
  static constexpr int P_OFF = Q_OFF + 16 * HD;                 // probabilities of two steps
  static constexpr int P_B = 2 * STEP * 32 * 8;
  static constexpr int RED_OFF = P_OFF + P_B;                   // partial O of warps that share a piece
  static constexpr int SMEM_B = RED_OFF + (KS > 1 ? kHeads * HD * KS * 4 : 0);
  static_assert(MINB * (SMEM_B + 1024 + 1024) <= 227 * 1024, "shared memory of the resident CTAs");
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

// Keys and records of one sequence.
struct Kv4Seq {
  int L, kbeg, first, n;  // visible keys [kbeg, L) in records [first, first + n)
};
__device__ __forceinline__ Kv4Seq seq_of_len(const Kv4DecodeArgs& a, int len) {
  Kv4Seq s;
  s.L = min(max(len, 0), a.len_cap);
  s.kbeg = a.window > 0 ? max(0, s.L - a.window) : 0;
  s.first = s.kbeg >> 4;
  s.n = ((s.L - 1) >> 4) + 1 - s.first;  // (none if L is 0)
  return s;
}

// (Lengths are read past L1, which may hold what they were before the wait.)
__device__ __forceinline__ Kv4Seq seq_of(const Kv4DecodeArgs& a, int b) { return seq_of_len(a, __ldcg(a.lens + b)); }

// The slot of a unit's part i, left by CTA c_first + i: the second of its two
// where the unit begins, else the first.
__device__ __forceinline__ int part_slot(int c_first, int i) { return 2 * (c_first + i) + (i == 0 ? 1 : 0); }

// Merges n <= kFan parts first, first + step, ... of a unit into out, or with out
// null (un-normalised) into the slot of the first.  Every thread forms the weights
// itself, so that all its loads are in flight at once.  s_ml: 2 kHeads floats.
template <int HD, int W>
__device__ __forceinline__ void merge_parts(const Kv4DecodeArgs& a, int c_first, int first, int step, int n, int G,
                                            __nv_bfloat16* out, float* s_ml) {  // (W warps)
  const int row = G * HD / 4;  // float4 of a slot
#pragma unroll 1
  for (int idx = threadIdx.x; idx < row; idx += W * 32) {
    const int h = idx * 4 / HD;
    const float4* src = reinterpret_cast<const float4*>(a.ws_o) + idx;
    float2 ml[kFan];
    float4 v[kFan];
#pragma unroll
    for (int i = 0; i < kFan; ++i) {
      const int slot = part_slot(c_first, first + min(i, n - 1) * step);
      ml[i] = __ldcg(&a.ws_ml[slot * kHeads + h]);
      v[i] = __ldcg(src + static_cast<size_t>(slot) * row);
    }
    float M = kNoKey, l = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kFan; ++i) M = fmaxf(M, ml[i].x);
#pragma unroll
    for (int i = 0; i < kFan; ++i) {
      if (i < n) {
        const float w = ex2_approx(ml[i].x - M);
        l = fmaf(w, ml[i].y, l);
        acc[0] = fmaf(w, v[i].x, acc[0]);
        acc[1] = fmaf(w, v[i].y, acc[1]);
        acc[2] = fmaf(w, v[i].z, acc[2]);
        acc[3] = fmaf(w, v[i].w, acc[3]);
      }
    }
    if (out != nullptr) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const float f[4] = {acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv};
      store_elems<4>(out + idx * 4, f);
    } else {
      store_elems<4>(a.ws_o + static_cast<size_t>(part_slot(c_first, first)) * G * HD + idx * 4, acc);
      if (idx * 4 % HD == 0) {
        s_ml[h] = M;
        s_ml[kHeads + h] = l;
      }
    }
  }
  if (out == nullptr) {  // (the first part's M and l are overwritten once every thread has read them)
    asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory");
    if (static_cast<int>(threadIdx.x) < G)
      a.ws_ml[part_slot(c_first, first) * kHeads + threadIdx.x] = make_float2(s_ml[threadIdx.x], s_ml[kHeads + threadIdx.x]);
  }
}

// A place in the units laid end to end: `off` records into (b, kvh), whose
// sequence has n records from `first` on; `left` records of the share remain.
struct Kv4Place {
  int b, kvh, off, left, first, n, L;
};

// GM: most heads per kv head, 4 (two scale blocks per product) or 8.
template <int HD, int GM>
__global__ void __launch_bounds__(Kv4Cfg<HD>::NT, Kv4Cfg<HD>::MINB)
    kv4_decode_kernel(const __grid_constant__ Kv4DecodeArgs a) {
  using C = Kv4Cfg<HD>;
  constexpr int RW = C::RW, STEP = C::STEP, PW = C::PW, KS = C::KS;
  constexpr int W = C::W, NT = C::NT, SLOTS = C::SLOTS;
  constexpr bool PAIR = GM == 4;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_bar[SLOTS];
  __shared__ long long s_scan[W + 1];
  __shared__ long long s_unit0;                      // records before the consumer's unit
  __shared__ Kv4Place s_ip, s_cp;                    // next step to copy; unit being consumed
  __shared__ float s_qf[kHeads];                     // score factor of each head
  __shared__ float s_top[W * kHeads];
  __shared__ float s_l[W * kHeads];
  __shared__ uint32_t s_ok[4];                       // records present in a step (step mod 4)
  __shared__ int s_c_first, s_nparts;                // cut at units: the unit's first CTA and parts
  __shared__ int s_last;
  __shared__ int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = a.H / a.Hkv;
  const int h0 = PAIR ? 2 * (t & 1) : 2 * t;               // this lane's columns are heads h0 and h0 + 1
  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) mbar_init(smem_u32(&s_bar[i]), 1);
    fence_mbar_init();
    s_abort = 0;
  }
  // ---- this CTA's share.  Formed before the wait from the lengths as they stand
  // (a batch of at most a sequence per thread), while the kernel before this one
  // finishes; after the wait it stands if no length has changed, else it is
  // formed again.  Nothing else is read before the wait, nothing written.
  const int per = (a.B + NT - 1) / NT;  // consecutive sequences per thread
  const int sb0 = min(a.B, tid * per), sb1 = min(a.B, sb0 + per);
  // exclusive sum of x over the threads, and its total
  auto scan = [&](long long x, long long& total) {
    long long upto = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w <= W; ++w) {
      if (w < warp) upto += s_scan[w];
      total += s_scan[w];
    }
    __syncthreads();
    return upto - x;
  };
  const int nctas = gridDim.x;
  const long long cta = blockIdx.x;
  const long long units = static_cast<long long>(a.B) * a.Hkv;
  auto steps_up = [](long long n) { return (n + STEP - 1) / STEP * STEP; };
  long long share = 0;
  bool cut_units = false;
  const bool one_each = per <= 1;
  int my_len = 0;  // one_each: this thread's sequence's
  auto my_seq = [&](int b) { return one_each ? seq_of_len(a, my_len) : seq_of(a, b); };
  auto read_len = [&] { return sb0 < sb1 ? __ldcg(a.lens + sb0) : 0; };
  // Sets share, cut_units and, where this CTA has work, the places; false if it has none.
  auto form_share = [&]() -> bool {
    long long sum = 0, total, at;
    for (int b = sb0; b < sb1; ++b) sum += my_seq(b).n;
    at = scan(sum, total) * a.Hkv;  // records before this thread's sequences
    total *= a.Hkv;
    share = steps_up((total + nctas - 1) / nctas);
    // Cut at every unit: parts of `cut` records (the last of a unit fewer), which
    // are at most total / cut + units; or as many as units, where no unit is longer.
    const int span = a.window > 0 && a.window < a.len_cap ? a.window : a.len_cap;
    const long long longest = steps_up((span + 15) / 16 + 1);
    const long long cut = nctas > units ? min(longest, steps_up((total + nctas - units - 1) / (nctas - units))) : 0;
    cut_units = cut > 0 && cut <= share + kCutSteps * STEP;
    Kv4Place p;  // where the share begins, set by the thread that finds it there
    p.left = 0;
    auto set = [&](int b, const Kv4Seq& seq, long long kvh, long long off, long long left) {
      p.b = b;
      p.kvh = static_cast<int>(kvh);
      p.off = static_cast<int>(off);
      p.left = static_cast<int>(left);
      p.first = seq.first;
      p.n = seq.n;
      p.L = seq.L;
    };
    bool work;
    if (cut_units) {
      long long parts = 0, nparts;
      for (int b = sb0; b < sb1; ++b) parts += (my_seq(b).n + cut - 1) / cut;
      long long before = scan(parts, nparts) * a.Hkv;
      work = cta < nparts * a.Hkv;
      if (cta >= before && cta < before + parts * a.Hkv) {
        for (int b = sb0; b < sb1; ++b) {
          const Kv4Seq seq = my_seq(b);
          const int np = static_cast<int>((seq.n + cut - 1) / cut);
          if (cta < before + static_cast<long long>(np) * a.Hkv) {
            const int rank = static_cast<int>(cta - before), part = rank % np;
            set(b, seq, rank / np, part * cut, min(cut, seq.n - part * cut));
            s_c_first = static_cast<int>(cta) - part;
            s_nparts = np;
            break;
          }
          before += static_cast<long long>(np) * a.Hkv;
        }
      }
    } else {
      const long long w0 = min(total, share * cta), w1 = min(total, w0 + share);
      work = w0 < w1;
      if (work && w0 >= at && w0 < at + sum * a.Hkv) {
        for (int b = sb0; b < sb1; ++b) {
          const Kv4Seq seq = my_seq(b);
          const long long n = seq.n;
          if (w0 < at + n * a.Hkv) {
            const long long kvh = (w0 - at) / n;
            set(b, seq, kvh, w0 - at - kvh * n, w1 - w0);
            s_unit0 = at + kvh * n;
            break;
          }
          at += n * a.Hkv;
        }
      }
    }
    if (p.left > 0) s_ip = s_cp = p;
    __syncthreads();
    return work;
  };
  bool work = false;
  if (one_each) {
    my_len = read_len();
    work = form_share();
  }
  pdl_wait();
  pdl_trigger();
  bool again = !one_each;
  if (one_each) {
    const int len = read_len();
    again = __syncthreads_or(len != my_len);
    my_len = len;
  }
  if (again) work = form_share();
  // sequences without keys, spread over the CTAs
  for (int b = blockIdx.x; b < a.B; b += nctas) {
    if (seq_of(a, b).n == 0) {
      uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<size_t>(b) * a.H * HD);
      for (int i = tid; i < a.H * HD / 2; i += NT) o[i] = 0u;
    }
  }
  if (!work) return;
  // Moves a place n records on within its unit, or to the next unit that has any.
  auto advance = [&](Kv4Place& p, int n) {
    p.off += n;
    p.left -= n;
    if (p.left <= 0 || p.off < p.n) return;
    p.off = 0;
    if (++p.kvh < a.Hkv) return;
    p.kvh = 0;
    Kv4Seq seq;
    do {  // (work is left, so a later sequence has records)
      seq = seq_of(a, ++p.b);
    } while (seq.n == 0);
    p.first = seq.first;
    p.n = seq.n;
    p.L = seq.L;
  };

  // The computing warps' barrier.
  auto sync_compute = [] { asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory"); };

  if (warp == W) {
    // ---- copies (warp W): part n = 2 step + (V ? 1 : 0) goes to buffer n mod SLOTS
    // once part n - SLOTS has been read; lane r < STEP copies record r of a step.
    // Block ids are loaded 32 records (of one unit) at a time, a batch ahead.
    int id = -1, id_next = -1;      // of the batch's record `lane`
    int n_batch = 0, n_next = 0, at_batch = 0;
    uint32_t rec = 0, rec_next = 0;  // its record's index among its head's in the block, kvh above
    const int rec_bits = a.block_shift - 4;
    auto load_batch = [&]() {  // the batch at s_ip; moves it past the batch
      Kv4Place p = s_ip;
      __syncwarp();
      id_next = -1;
      n_next = 0;
      if (p.left <= 0) return;
      const int n = min(min(32, p.n - p.off), p.left);
      if (lane < n) {
        const int gi = p.first + p.off + lane;
        const int entry = gi >> rec_bits;
        if (entry < a.max_blocks) id_next = a.table[static_cast<size_t>(p.b) * a.max_blocks + entry];
        rec_next = static_cast<uint32_t>(p.kvh) << rec_bits | (gi & ((1 << rec_bits) - 1));
      }
      n_next = n;
      advance(p, n);
      if (lane == 0) s_ip = p;
      __syncwarp();
    };
    int issued = 0, copied = 0;  // parts
    int id_k = -1;   // of the step being issued
    uint32_t rec_k = 0;
    auto issue = [&]() -> bool {  // part `issued`, if there is one
      const bool is_v = issued & 1;
      if (!is_v) {
        if (at_batch >= n_batch) {
          id = id_next;
          rec = rec_next;
          n_batch = n_next;
          at_batch = 0;
          load_batch();
        }
        if (n_batch == 0) return false;
        id_k = __shfl_sync(0xffffffffu, id, at_batch + lane);
        rec_k = __shfl_sync(0xffffffffu, rec, at_batch + lane);
        if (lane >= STEP || at_batch + lane >= n_batch || id_k >= a.n_blocks) id_k = -1;
        at_batch += STEP;
      }
      // (after an abandoned wait the steps are only counted)
      if (!__any_sync(0xffffffffu, *static_cast<volatile int*>(&s_abort))) {
        const uint32_t bar = smem_u32(&s_bar[issued % SLOTS]);
        const uint32_t all = __ballot_sync(0xffffffffu, id_k >= 0);
        if (lane == 0) {
          if (!is_v) s_ok[(issued >> 1) & 3] = all;
          mbar_arrive_expect_tx(bar, __popc(all) * C::HALF_B);
        }
        __syncwarp();
        if (id_k >= 0) {
          const size_t r = (static_cast<size_t>(id_k) * a.Hkv << rec_bits) + rec_k;
          bulk_g2s(smem_u32(smem) + (issued % SLOTS) * C::SLOT_B + lane * C::HALF_B,
                   a.data + r * Kv4Rec<HD>::BYTES + (is_v ? C::HALF_B : 0), C::HALF_B, bar);
        }
        copied = issued + 1;
      }
      ++issued;
      return true;
    };
    load_batch();
    int ready = 0;  // parts issued so far
#pragma unroll 1
    for (int i = 0; i < SLOTS && issue(); ++i) ++ready;
    // One CTA barrier per step: then the step's K buffer and the last step's V
    // buffer are free.
#pragma unroll 1
    for (int k = 0; 2 * k < ready; ++k) {
      __syncthreads_or(0);
      if (k > 0 && issue()) ++ready;
      if (issue()) ++ready;
    }
    // After an abandoned wait: the copies still in flight.
    if (*static_cast<volatile int*>(&s_abort)) {
      for (int n = max(0, copied - SLOTS); n < copied; ++n)
        warp_wait(smem_u32(&s_bar[n % SLOTS]), (n / SLOTS) & 1, nullptr);
    }
    return;
  }

  const int qrec = warp * RW;                              // first record this warp scores
  const int vpiece = KS > 1 ? (warp % C::NP) : warp * PW;  // first piece of O of this warp
  const int vrec0 = KS > 1 ? warp / C::NP : 0;             // its records of a step: vrec0, vrec0 + KS, ...

  // s += the products of 64 elements of a record's keys with q
  auto score_piece = [&](float (&s)[4], const uint8_t* rec, int p) {
    const uint4 kc = *reinterpret_cast<const uint4*>(rec + p * 512 + lane * 16);
    const uint4 qa = *reinterpret_cast<const uint4*>(smem + C::Q_OFF + ((2 * p) * 32 + lane) * 16);
    const uint4 qb = *reinterpret_cast<const uint4*>(smem + C::Q_OFF + ((2 * p + 1) * 32 + lane) * 16);
    auto scale_add = [&](uint32_t f16s, const float (&d)[4]) {
      const float2 sc = __half22float2(as_half2(f16s));
      s[0] = fmaf(sc.x, d[0], s[0]);
      s[1] = fmaf(sc.x, d[1], s[1]);
      s[2] = fmaf(sc.y, d[2], s[2]);
      s[3] = fmaf(sc.y, d[3], s[3]);
    };
    if constexpr (PAIR) {
      const uint8_t* ks = rec + 8 * HD + p * 64 + g * 8 + (t >> 1) * 2;  // block 2j + (t >> 1): columns 0-3, 4-7
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t c0 = j ? kc.y : kc.x, c1 = j ? kc.w : kc.z;
        const uint4 q = j ? qb : qa;
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        mma_f16(d, e2m1x2_f16x2<0>(c0), e2m1x2_f16x2<0>(c1), e2m1x2_f16x2<2>(c0), e2m1x2_f16x2<2>(c1), q.x, q.y);
        mma_f16(d, e2m1x2_f16x2<1>(c0), e2m1x2_f16x2<1>(c1), e2m1x2_f16x2<3>(c0), e2m1x2_f16x2<3>(c1), q.z, q.w);
        scale_add(e4m3x2_f16x2(*reinterpret_cast<const uint16_t*>(ks + j * 4)), d);
      }
    } else {
      const uint2 ks = *reinterpret_cast<const uint2*>(rec + 8 * HD + p * 64 + g * 8);
      const uint32_t qw[8] = {qa.x, qa.y, qa.z, qa.w, qb.x, qb.y, qb.z, qb.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t c0 = w < 2 ? kc.x : kc.y, c1 = w < 2 ? kc.z : kc.w;
        const uint32_t sw = w < 2 ? ks.x : ks.y;
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (w & 1)
          mma_f16(d, e2m1x2_f16x2<2>(c0), e2m1x2_f16x2<2>(c1), e2m1x2_f16x2<3>(c0), e2m1x2_f16x2<3>(c1), qw[2 * w],
                  qw[2 * w + 1]);
        else
          mma_f16(d, e2m1x2_f16x2<0>(c0), e2m1x2_f16x2<0>(c1), e2m1x2_f16x2<1>(c0), e2m1x2_f16x2<1>(c1), qw[2 * w],
                  qw[2 * w + 1]);
        scale_add(w & 1 ? e4m3x2_hi_f16x2(sw) : e4m3x2_f16x2(sw), d);
      }
    }
  };
  // O^T += V^T (P s)^T for 64 elements of a record's values
  auto add_piece = [&](float (*o)[4], const uint8_t* rec, int p, uint2 pp) {
    const uint4 vc = *reinterpret_cast<const uint4*>(rec + p * 512 + lane * 16);
    const __half2 pa = as_half2(pp.x), pb = as_half2(pp.y);
    // pairs of positions side by side, for the even and the odd elements
    const uint32_t lo01 = (vc.x & 0x0f0f0f0fu) | ((vc.y << 4) & 0xf0f0f0f0u);
    const uint32_t hi01 = ((vc.x >> 4) & 0x0f0f0f0fu) | (vc.y & 0xf0f0f0f0u);
    const uint32_t lo23 = (vc.z & 0x0f0f0f0fu) | ((vc.w << 4) & 0xf0f0f0f0u);
    const uint32_t hi23 = ((vc.z >> 4) & 0x0f0f0f0fu) | (vc.w & 0xf0f0f0f0u);
    const uint8_t* vs = rec + 8 * HD + p * 64 + t * 16;
    if constexpr (PAIR) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t sw = *reinterpret_cast<const uint32_t*>(vs + (2 * j + (g >> 2)) * 4);
        const uint32_t b0 = as_u32(__hmul2(pa, as_half2(e4m3x2_f16x2(sw))));
        const uint32_t b1 = as_u32(__hmul2(pb, as_half2(e4m3x2_hi_f16x2(sw))));
        if (j == 0) {
          mma_f16(o[0], e2m1x2_f16x2<0>(lo01), e2m1x2_f16x2<1>(lo01), e2m1x2_f16x2<0>(lo23), e2m1x2_f16x2<1>(lo23), b0, b1);
          mma_f16(o[1], e2m1x2_f16x2<0>(hi01), e2m1x2_f16x2<1>(hi01), e2m1x2_f16x2<0>(hi23), e2m1x2_f16x2<1>(hi23), b0, b1);
        } else {
          mma_f16(o[2], e2m1x2_f16x2<2>(lo01), e2m1x2_f16x2<3>(lo01), e2m1x2_f16x2<2>(lo23), e2m1x2_f16x2<3>(lo23), b0, b1);
          mma_f16(o[3], e2m1x2_f16x2<2>(hi01), e2m1x2_f16x2<3>(hi01), e2m1x2_f16x2<2>(hi23), e2m1x2_f16x2<3>(hi23), b0, b1);
        }
      }
    } else {
      const uint4 v4 = *reinterpret_cast<const uint4*>(vs);
      const uint32_t vsw[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t b0 = as_u32(__hmul2(pa, as_half2(e4m3x2_f16x2(vsw[w]))));
        const uint32_t b1 = as_u32(__hmul2(pb, as_half2(e4m3x2_hi_f16x2(vsw[w]))));
        switch (w) {
          case 0: mma_f16(o[0], e2m1x2_f16x2<0>(lo01), e2m1x2_f16x2<0>(hi01), e2m1x2_f16x2<0>(lo23), e2m1x2_f16x2<0>(hi23), b0, b1); break;
          case 1: mma_f16(o[1], e2m1x2_f16x2<1>(lo01), e2m1x2_f16x2<1>(hi01), e2m1x2_f16x2<1>(lo23), e2m1x2_f16x2<1>(hi23), b0, b1); break;
          case 2: mma_f16(o[2], e2m1x2_f16x2<2>(lo01), e2m1x2_f16x2<2>(hi01), e2m1x2_f16x2<2>(lo23), e2m1x2_f16x2<2>(hi23), b0, b1); break;
          default: mma_f16(o[3], e2m1x2_f16x2<3>(lo01), e2m1x2_f16x2<3>(hi01), e2m1x2_f16x2<3>(lo23), e2m1x2_f16x2<3>(hi23), b0, b1); break;
        }
      }
    }
  };
  // The output of this lane's x-th of 2 PW element pairs: elements d, d + 1 (of
  // the head) of heads h0 and h0 + 1.
  auto out_pairs = [&](float (*o)[4], auto&& put) {
#pragma unroll
    for (int x = 0; x < PW * 4; ++x) {
      if constexpr (PAIR) {  // products 2j and 2j + 1: even and odd elements of block 2j (t < 2) or 2j + 1
        if (x & 1) continue;
        const int d = vpiece * 64 + (x + (t >> 1)) * 16 + 2 * g;
        const bool up = t >= 2;
        put(d, make_float2(up ? o[x][2] : o[x][0], up ? o[x + 1][2] : o[x + 1][0]),
            make_float2(up ? o[x][3] : o[x][1], up ? o[x + 1][3] : o[x + 1][1]));
      } else {
        const int d = vpiece * 64 + x * 16 + 2 * g;
        put(d, make_float2(o[x][0], o[x][2]), make_float2(o[x][1], o[x][3]));
      }
    }
  };
  // The parts in turn: buffer and parity of the next one.
  int slot = 0;
  uint32_t parity = 0;
  auto wait_part = [&](const uint8_t*& part) {
    part = smem + slot * C::SLOT_B;
    const bool ok = warp_wait(smem_u32(&s_bar[slot]), parity, a.err, &s_abort);
    if (++slot == SLOTS) {
      slot = 0;
      parity ^= 1;
    }
    return ok;
  };

  int k = 0;  // step of the share
  while (true) {
    // ---- a unit (or the part of one in this share) begins
    const int r0 = s_cp.first + s_cp.off;                  // first record
    const int nrec = min(s_cp.n - s_cp.off, s_cp.left);
    const int L = s_cp.L, kbeg = seq_of_len(a, L).kbeg;
    // q fragments: lane (column g, t) holds elements 4t .. 4t+3 of every 16, two
    // blocks side by side, zeros in columns without a head (and, two blocks to a
    // product, where the other block's elements stand); each head scaled by the
    // power of two that brings its largest element into [1, 2).
    {
      const __nv_bfloat16* q =
          static_cast<const __nv_bfloat16*>(a.q) + (static_cast<size_t>(s_cp.b) * a.H + s_cp.kvh * G) * HD;
#pragma unroll 1
      for (int h = warp; h < GM; h += W) {
        constexpr int PER = HD / 32;  // elements per lane, consecutive
        float x[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) x[i] = 0.0f;
        if (h < G) load_elems<PER>(q + h * HD + lane * PER, x);
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
        for (int x2 = 16; x2 > 0; x2 >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x2));
        int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        e = top > 0.0f ? min(max(e, -120), 120) : 0;
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        if (lane == 0) s_qf[h] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
        for (int i = 0; i < PER; i += 2) {
          const int d = lane * PER + i;
          const int blk = d >> 4, tt = (d >> 2) & 3, odd = (d >> 1) & 1;  // odd: elements 4t+2, 4t+3
          const uint32_t v = pack_f16x2(x[i] * down, x[i + 1] * down);
          uint32_t* at = reinterpret_cast<uint32_t*>(smem + C::Q_OFF + (blk >> 1) * 512);
          if constexpr (PAIR) {  // column h + 4 (block 2j + 1), words {product 1: b0, b1; product 2: b0, b1}
            const int up = blk & 1;
            *reinterpret_cast<uint2*>(at + ((h + 4 * up) * 4 + tt) * 4 + odd * 2) = up ? make_uint2(0u, v) : make_uint2(v, 0u);
          } else {
            at[(h * 4 + tt) * 4 + (blk & 1) * 2 + odd] = v;
          }
        }
      }
    }
    float o[PW * 4][4];
#pragma unroll
    for (int i = 0; i < PW * 4; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m0 = kNoKey, m1 = kNoKey, l0 = 0.0f, l1 = 0.0f;  // heads h0 and h0 + 1
    sync_compute();
    const float qf0 = s_qf[h0], qf1 = s_qf[h0 + 1];

#pragma unroll 1
    for (int done = 0; done < nrec; done += STEP, ++k) {
      const int base = r0 + done, nhere = min(STEP, nrec - done);
      // a step that lies wholly inside [kbeg, L) and the share needs no masks
      const bool edge = base * kKv4Group < kbeg || (base + STEP) * kKv4Group > L || nhere < STEP;
      // ---- scores of this warp's records
      float s[RW][4];
#pragma unroll
      for (int i = 0; i < RW; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
      const uint8_t* kpart;
      if (wait_part(kpart)) {
        kpart += qrec * C::HALF_B;
#pragma unroll
        for (int i = 0; i < RW; ++i) {
#pragma unroll
          for (int p = 0; p < C::NP; ++p) score_piece(s[i], kpart + i * C::HALF_B, p);
          if constexpr (PAIR) {  // the two blocks' columns
#pragma unroll
            for (int x = 0; x < 4; ++x) s[i][x] += __shfl_xor_sync(0xffffffffu, s[i][x], 2);
          }
        }
      }
      // ---- their probabilities
      float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        s[i][0] *= qf0;
        s[i][1] *= qf1;
        s[i][2] *= qf0;
        s[i][3] *= qf1;
        if (edge) {  // positions outside [kbeg, L), and records past the share: no weight
          const int pos = (base + qrec + i) * kKv4Group + g;
          const bool in = qrec + i < nhere;
          if (!in || pos < kbeg || pos >= L) s[i][0] = s[i][1] = -INFINITY;
          if (!in || pos + 8 < kbeg || pos + 8 >= L) s[i][2] = s[i][3] = -INFINITY;
        }
        top0 = fmaxf(top0, fmaxf(s[i][0], s[i][2]));
        top1 = fmaxf(top1, fmaxf(s[i][1], s[i][3]));
      }
      uint2* pbuf = reinterpret_cast<uint2*>(smem + C::P_OFF) + (k & 1) * STEP * 32;
      float ps0, ps1;
      auto probabilities = [&]() {
        const float ref0 = m0 - kShift, ref1 = m1 - kShift;
        ps0 = ps1 = 0.0f;
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          const float p0 = ex2_approx(s[i][0] - ref0), p1 = ex2_approx(s[i][1] - ref1);
          const float p2 = ex2_approx(s[i][2] - ref0), p3 = ex2_approx(s[i][3] - ref1);
          ps0 += p0 + p2;
          ps1 += p1 + p3;
          // head g; positions 2t, 2t+1 and 2t+8, 2t+9
          pbuf[(qrec + i) * 32 + lane] =
              make_uint2(transpose8x8(pack_f16x2(p0, p1)), transpose8x8(pack_f16x2(p2, p3)));
        }
      };
      probabilities();
      const bool any_over = __syncthreads_or(top0 > m0 + kSlack || top1 > m1 + kSlack);
      // A step with absent blocks (scored from whatever their buffers hold) or
      // with scores far above the reference is weighed again.
      const uint32_t ok = s_ok[k & 3];
      const bool gaps = ok != (1u << nhere) - 1u;
      if (any_over || gaps) {
        top0 = top1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          if (!((ok >> (qrec + i)) & 1u)) s[i][0] = s[i][1] = s[i][2] = s[i][3] = -INFINITY;
          top0 = fmaxf(top0, fmaxf(s[i][0], s[i][2]));
          top1 = fmaxf(top1, fmaxf(s[i][1], s[i][3]));
        }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, x));
          top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, x));
        }
        if (g == 0) {
          s_top[warp * kHeads + 2 * t] = top0;
          s_top[warp * kHeads + 2 * t + 1] = top1;
        }
        sync_compute();
        float n0 = m0, n1 = m1;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          n0 = fmaxf(n0, s_top[w * kHeads + 2 * t]);
          n1 = fmaxf(n1, s_top[w * kHeads + 2 * t + 1]);
        }
        const float f0 = ex2_approx(m0 - n0), f1 = ex2_approx(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int x = 0; x < PW * 4; ++x) {
          o[x][0] *= f0;
          o[x][1] *= f1;
          o[x][2] *= f0;
          o[x][3] *= f1;
        }
        probabilities();
        sync_compute();
      }
      l0 += ps0;
      l1 += ps1;

      // ---- P V of the step for this warp's pieces
      const uint8_t* vpart;
      const bool vthere = wait_part(vpart);
      if (edge || gaps) {
        // V scales of positions outside [kbeg, L) and of absent records may be
        // any bytes, even NaN: each warp zeroes those of the records it scored.
#pragma unroll
        for (int i = qrec; i < qrec + RW; ++i) {
          uint32_t* vs = reinterpret_cast<uint32_t*>(const_cast<uint8_t*>(vpart) + i * C::HALF_B + 8 * HD);
          for (int x = lane; x < HD / 4; x += 32) {
            const int m = (base + i) * kKv4Group + 2 * ((x >> 2) & 3);  // the word's positions: m, m + 1, m + 8, m + 9
            auto seen = [&](int pos) { return pos >= kbeg && pos < L; };
            const uint32_t mask = (seen(m) ? 0xffu : 0u) | (seen(m + 1) ? 0xff00u : 0u) |
                                  (seen(m + 8) ? 0xff0000u : 0u) | (seen(m + 9) ? 0xff000000u : 0u);
            vs[x] = (ok >> i) & 1u ? vs[x] & mask : 0u;
          }
        }
        fence_proxy_async_smem();  // (the next copy into this buffer comes after these stores)
        sync_compute();
      }
      if (vthere) {
#pragma unroll
        for (int ii = 0; ii < STEP / KS; ++ii) {
          const int i = vrec0 + ii * KS;
          const uint2 pp = pbuf[i * 32 + lane];
#pragma unroll
          for (int pi = 0; pi < PW; ++pi) add_piece(o + pi * 4, vpart + i * C::HALF_B, vpiece + pi, pp);
        }
      }
    }

    // ---- the unit's part in this share ends
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, x);
      l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
    if (g == 0) {
      s_l[warp * kHeads + 2 * t] = l0;
      s_l[warp * kHeads + 2 * t + 1] = l1;
    }
    float* red = reinterpret_cast<float*>(smem + C::RED_OFF);  // [KS][head][HD]
    if constexpr (KS > 1) {
      if (vrec0 > 0)
        out_pairs(o, [&](int d, float2 u, float2 v) {
          float* r = red + vrec0 * kHeads * HD + d;
          *reinterpret_cast<float2*>(r + h0 * HD) = u;
          *reinterpret_cast<float2*>(r + (h0 + 1) * HD) = v;
        });
    }
    sync_compute();
    l0 = l1 = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      l0 += s_l[w * kHeads + h0];
      l1 += s_l[w * kHeads + h0 + 1];
    }
    const Kv4Place cp = s_cp;
    const long long unit0 = s_unit0;
    const int c_first = cut_units ? s_c_first : static_cast<int>(unit0 / share);
    const int nparts = cut_units ? s_nparts : static_cast<int>((unit0 + cp.n - 1) / share) - c_first + 1;
    const bool whole = nparts == 1;
    const int place = part_slot(c_first, static_cast<int>(blockIdx.x) - c_first);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (static_cast<size_t>(cp.b) * a.H + cp.kvh * G) * HD;
    if (vrec0 == 0) {
      // (l is zero only where no key was present; a NaN stays one)
      const float i0 = l0 == 0.0f ? 0.0f : 1.0f / l0, i1 = l1 == 0.0f ? 0.0f : 1.0f / l1;
      out_pairs(o, [&](int d, float2 u, float2 v) {
        if constexpr (KS > 1) {
#pragma unroll
          for (int y = 1; y < KS; ++y) {
            const float* r = red + y * kHeads * HD + d;
            const float2 ru = *reinterpret_cast<const float2*>(r + h0 * HD);
            const float2 rv = *reinterpret_cast<const float2*>(r + (h0 + 1) * HD);
            u.x += ru.x;
            u.y += ru.y;
            v.x += rv.x;
            v.y += rv.y;
          }
        }
        if (whole) {
          if (h0 < G) *reinterpret_cast<uint32_t*>(out + h0 * HD + d) = pack_bf16x2(u.x * i0, u.y * i0);
          if (h0 + 1 < G) *reinterpret_cast<uint32_t*>(out + (h0 + 1) * HD + d) = pack_bf16x2(v.x * i1, v.y * i1);
        } else {
          float* w = a.ws_o + static_cast<size_t>(place) * G * HD + d;
          if (h0 < G) *reinterpret_cast<float2*>(w + h0 * HD) = u;
          if (h0 + 1 < G) *reinterpret_cast<float2*>(w + (h0 + 1) * HD) = v;
        }
      });
    }
    if (!whole) {
      if (warp == 0 && g == 0) {
        if (h0 < G) a.ws_ml[place * kHeads + h0] = make_float2(m0, l0);
        if (h0 + 1 < G) a.ws_ml[place * kHeads + h0 + 1] = make_float2(m1, l1);
      }
      // Parts are merged kFan neighbours at a time by the CTA that completes them,
      // each merge left in the slot of its first part, until one is left.
      int part = static_cast<int>(blockIdx.x) - c_first, left = nparts, step = 1;
      unsigned* tickets = a.tickets;  // [level][slot of a merge's first part]
#pragma unroll 1
      while (true) {
        const int first = part / kFan * kFan, n = min(kFan, left - first);
        unsigned* ticket = tickets + part_slot(c_first, first * step);
        __threadfence();
        sync_compute();
        if (tid == 0) {
          s_last = atomicAdd(ticket, 1u) == static_cast<unsigned>(n - 1);
          if (s_last) *ticket = 0u;  // ready for the next call
        }
        sync_compute();
        if (!s_last) break;
        __threadfence();
        const bool final = left <= kFan;
        merge_parts<HD, W>(a, c_first, first * step, step, n, G, final ? out : nullptr, s_top);
        if (final) break;
        part /= kFan;
        left = (left + kFan - 1) / kFan;
        step *= kFan;
        tickets += 2 * kKv4MaxCtas;
      }
    }
    if (cp.left <= nrec) break;
    sync_compute();  // (every thread has read the place)
    if (tid == 0) {
      Kv4Place p = cp;
      advance(p, nrec);
      s_unit0 = unit0 + cp.n;
      s_cp = p;
    }
    sync_compute();
  }
}

template <int HD, int GM>
cudaError_t launch_hg(const Kv4DecodeArgs& a, cudaStream_t s) {
  using C = Kv4Cfg<HD>;
  const cudaError_t e = set_smem_limit_once<kv4_decode_kernel<HD, GM>>(C::SMEM_B);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.nctas));
  cfg.blockDim = dim3(C::NT);
  cfg.dynamicSmemBytes = C::SMEM_B;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_decode_kernel<HD, GM>, a);
}

template <int HD>
cudaError_t launch_h(const Kv4DecodeArgs& a, cudaStream_t s) {
  // Up to 4 heads: two scale blocks per product (133 us against 152 with one at head_dim
  // 512, 4 x 131072 keys, before the copies had a warp of their own).
  if (a.H <= 4 * a.Hkv) return launch_hg<HD, 4>(a, s);
  if constexpr (HD <= 256) return launch_hg<HD, 8>(a, s);
  return cudaErrorInvalidValue;
}

template <int HD>
Kv4DecodePlan plan_h(int window, int H, int Hkv, int B, int max_seq_len) {
  using C = Kv4Cfg<HD>;
  const int span = window > 0 && window < max_seq_len ? window : max_seq_len;
  // a window that starts inside a record touches one more
  const long long groups = (static_cast<long long>(span) + 15) / 16 + (span < max_seq_len ? 1 : 0);
  const long long units = static_cast<long long>(B) * Hkv;
  // as many CTAs as are resident, each with a step or more
  long long n = units * ((groups + C::STEP - 1) / C::STEP + 1);
  const long long slots = static_cast<long long>(sm_count()) * C::MINB;
  if (n > slots) n = slots;
  static_assert(kKv4MaxCtas <= kFan * kFan * kFan * kFan, "levels of merges");
  if (n > kKv4MaxCtas) n = kKv4MaxCtas;
  Kv4DecodePlan p;
  p.nctas = static_cast<int>(n);
  const size_t G = static_cast<size_t>(H / Hkv);
  p.o_bytes = (2 * static_cast<size_t>(n) * G * HD * 4 + 255) / 256 * 256;
  p.ml_bytes = (2 * static_cast<size_t>(n) * kHeads * 8 + 255) / 256 * 256;
  p.ws_bytes = n > 1 ? kKv4TicketBytes + p.ml_bytes + p.o_bytes : 0;
  return p;
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
  switch (hd) {
    case 64: return plan_h<64>(window, H, Hkv, B, max_seq_len);
    case 128: return plan_h<128>(window, H, Hkv, B, max_seq_len);
    case 256: return plan_h<256>(window, H, Hkv, B, max_seq_len);
    default: return plan_h<512>(window, H, Hkv, B, max_seq_len);
  }
}

}  // namespace g4
