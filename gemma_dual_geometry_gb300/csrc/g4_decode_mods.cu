// Decode attention with modified scores (g4_attn_decode_mods): one query per
// sequence over the bf16 or float32 cache, HBM-bound.
//
//   out_h = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),  s = c tanh(scale q.k / c) -
//   slope_h (L - 1 - j) in log2 units, over the keys [max(key_begin, L - window), L).
//
// Work.  The keys of all (sequence, kv head) units, laid end to end, are dealt out in
// equal contiguous shares to as many CTAs as are resident, so that lengths of all
// sizes, and sequences that begin late in their cache, leave no SM idle.  Where
// that makes no share much longer, shares are cut anew at every unit instead, so
// that no CTA pays for the start of a second one.  A unit inside one share is
// written directly; the parts of one that spans shares meet in the workspace, where
// the CTA that completes kFan neighbours merges them, level by level, until one is left.
//
// A share's keys go through the CTA as in g4_attn_simt.cuh: stages of a few rows
// to the warps in turn, each with its own ring of bulk copies, the G heads of the
// kv head sharing every row, a cap and a bias applied in the lane that holds a score.
//
// Measured (device time; copy rate 6.78 TB/s): head_dim 512, 8 heads on 2, 64 sequences
// of 1024 to 8192 keys, capped 197 us, 6.1 TB/s (237 with equal splits of the longest length); 4 of
// 131072 with a bias that begin anywhere 250 us, 5.8 TB/s (311); 8 of 4097 36 us, 3.7 TB/s.
// 64 sequences of 1024 to 8192 keys of 256 101 us, 6.0 TB/s; of 128 63 us, 4.8 TB/s.
//   What bounds it: at head_dim 512 and 256 with up to 4 heads per kv head, and with one or two at any, the bytes; otherwise
// instruction issue (each key's partial products are reduced over the warp); with few keys the start (lengths,
// scans, first copies) and the merges, some 10 us.
#include <math.h>

#include <algorithm>

#include "g4_attn_simt.cuh"

namespace g4 {
namespace {

// Parts merged at once.  8: 92 us against 81 at 64 sequences of 1024 to 8192 keys of head_dim 128 (8 heads on 2), 107
// against 98 at head_dim 64 (8 on 8), but 37.8 against 39.4 at 8 of 4097 keys of 512.
constexpr int kFan = 16;
constexpr int kLevels = 3;     // of merges
constexpr int kMaxCtas = 1024;
static_assert(kMaxCtas <= kFan * kFan * kFan, "levels of merges");
// The counters have a place of their own whatever the call, so that a workspace may serve any call after any other.
constexpr size_t kTicketBytes = kLevels * 2 * kMaxCtas * sizeof(unsigned);
constexpr int kMinShare = 64;  // keys per CTA, at least
// Shares are cut at units where that makes the longest one at most an eighth longer.
constexpr int kCutShift = 3;

// The slot of a unit's part i, left by CTA c_first + i: the second of its two
// where the unit begins, else the first.
__device__ __forceinline__ int part_slot(int c_first, int i) { return 2 * (c_first + i) + (i == 0 ? 1 : 0); }

// CTAs per SM: two where q and O of the group take some 180 registers of a thread, three otherwise; four for rows of up to
// 256 bytes, whose stages are short (64 x 1024 .. 8192 keys, four against three, with batches of 16: head_dim 128, 4 heads
// 74 us against 81, head_dim 64 93 against 97; head_dim 256, 2 heads 219 against 184; five or six are slower throughout).
constexpr int resident_ctas(int warps, int group_width, int row_bytes) {
  return warps > 4 ? 1 : group_width >= 2048 ? 2 : group_width > 512 || row_bytes > 256 ? 3 : 4;
}

// Scores that a warp sums over its lanes at a time, for rows of ROWB bytes.  32 where they are short: every lane has a
// score of its own, and twice the keys share a batch's fixed costs (64 x 1024 .. 8192 keys, 32 against 16: head_dim 128, 4
// heads per kv head 63 us against 74, 8 heads 105 against 128; head_dim 256, 4 heads 101 against 119, 8 heads 185 against 229;
// 256 windows of 512 keys of 256 57 against 65).  Rows of 1 KB would need stages of 8 KB, and so a CTA less per SM.
template <int ROWB>
constexpr int kBatch = ROWB <= 512 ? 32 : kNPMax;

// The keys of one sequence.
struct SeqKeys {
  int L, kbeg;  // [kbeg, L)
};
__device__ __forceinline__ SeqKeys seq_keys(const ModsDecodeArgs& a, int b) {
  SeqKeys s;
  s.L = min(max(__ldcg(a.lens + b), 0), a.len_cap);
  s.kbeg = a.window > 0 ? max(0, s.L - a.window) : 0;
  if (a.key_begin != nullptr) s.kbeg = min(max(s.kbeg, __ldcg(a.key_begin + b)), s.L);
  return s;
}

// A run of one unit's keys: keys [k0, k1) of sequence b's kv head, part `part` of `nparts`; the first of them is
// CTA c_first's.
struct Run {
  int b, kvh, k0, k1, L, part, nparts;
};

// What follows the streaming area in shared memory.
template <int NW, int NST, int G>
struct Tail {
  uint64_t bars[NW * NST];
  long long scan[NW];
  long long unit0;           // keys before the run's unit
  Run run;
  float sc[NW][32];  // (kBatch, at most)
  float sa[NW][8];
  float ml[2][G];
  int last;
};

template <typename T, int HD, int G, int NW>
__global__ void __launch_bounds__(NW * 32, resident_ctas(NW, G * HD, HD * sizeof(T)))
    decode_mods_kernel(const __grid_constant__ ModsDecodeArgs a) {
  using C = SimtCfg<T, HD, G, NW, kBatch<HD * sizeof(T)>>;
  constexpr int EL2 = C::EL / 2;
  constexpr int NT = NW * 32;
  extern __shared__ __align__(1024) uint8_t smem[];
  Tail<NW, C::NST, G>& sh = *reinterpret_cast<Tail<NW, C::NST, G>*>(smem + C::AREA_B);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* wbar = sh.bars + warp * C::NST;
  if (lane == 0) {
    for (int i = 0; i < C::NST; ++i) mbar_init(smem_u32(&wbar[i]), 1);
    fence_mbar_init();
  }
  __syncwarp();

  // ---- this CTA's share.  Formed before the wait from the lengths as they stand (a batch of at most a sequence per
  // thread), while the kernel before this one finishes; after the wait it stands if nothing has changed, else it is
  // formed again.  Nothing else is read before the wait, nothing written.
  const int nctas = gridDim.x;
  const long long cta = blockIdx.x;
  const long long units = static_cast<long long>(a.B) * a.Hkv;
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
    if (lane == 31) sh.scan[warp] = upto;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) upto += sh.scan[w];
      total += sh.scan[w];
    }
    __syncthreads();
    return upto - x;
  };
  const bool one_each = per <= 1;
  SeqKeys mine = {0, 0};
  auto keys_of = [&](int b) { return one_each ? mine : seq_keys(a, b); };  // of one of this thread's sequences
  long long share = 0;
  long long left = 0;  // keys of the share that are left (equal shares)
  bool cut_units = false;
  // Sets share, left, cut_units and, where this CTA has work, sh.run; false if it has none.
  auto form_share = [&]() -> bool {
    long long sum = 0, total;
    for (int b = sb0; b < sb1; ++b) {
      const SeqKeys s = keys_of(b);
      sum += s.L - s.kbeg;
    }
    long long at = scan(sum, total) * a.Hkv;  // keys before this thread's sequences
    total *= a.Hkv;
    // (where there are units enough for all CTAs, starting them is the work)
    share = max(units < nctas ? static_cast<long long>(kMinShare) : 1LL, (total + nctas - 1) / nctas);
    // (with a CTA for every unit and none of more than kMinShare keys, 300 keys of 75 units were 5 shares: 42 us)
    const long long cut = nctas > units ? max(static_cast<long long>(kMinShare), (total + nctas - units - 1) / (nctas - units))
                          : nctas == units && (a.window > 0 ? min(a.window, a.len_cap) : a.len_cap) <= kMinShare ? kMinShare
                                                                                                                 : 0;
    cut_units = cut > 0 && cut <= share + (share >> kCutShift);
    if (cut_units) {
      // parts of `cut` keys, the last of a unit fewer: at most total / cut + units <= nctas of them
      long long parts = 0, nparts;
      for (int b = sb0; b < sb1; ++b) {
        const SeqKeys s = keys_of(b);
        parts += (s.L - s.kbeg + cut - 1) / cut;
      }
      long long before = scan(parts, nparts) * a.Hkv;
      if (cta >= before && cta < before + parts * a.Hkv) {
        for (int b = sb0; b < sb1; ++b) {
          const SeqKeys s = keys_of(b);
          const long long np = (s.L - s.kbeg + cut - 1) / cut;
          if (cta < before + np * a.Hkv) {
            const long long rank = cta - before, part = rank % np, k0 = s.kbeg + part * cut;
            sh.run = {b, static_cast<int>(rank / np), static_cast<int>(k0),
                      static_cast<int>(min(static_cast<long long>(s.L), k0 + cut)), s.L, static_cast<int>(part),
                      static_cast<int>(np)};
            break;
          }
          before += np * a.Hkv;
        }
      }
      return cta < nparts * a.Hkv;
    }
    const long long w0 = min(total, share * cta), w1 = min(total, w0 + share);
    left = w1 - w0;
    if (left > 0 && w0 >= at && w0 < at + sum * a.Hkv) {
      for (int b = sb0; b < sb1; ++b) {
        const SeqKeys s = keys_of(b);
        const long long n = s.L - s.kbeg;
        if (w0 < at + n * a.Hkv) {
          const long long kvh = (w0 - at) / n, unit0 = at + kvh * n, k0 = s.kbeg + (w0 - unit0);
          const long long c0 = unit0 / share, c1 = (unit0 + n - 1) / share;
          sh.run = {b, static_cast<int>(kvh), static_cast<int>(k0), static_cast<int>(min(static_cast<long long>(s.L), k0 + left)),
                    s.L, static_cast<int>(cta - c0), static_cast<int>(c1 - c0 + 1)};
          sh.unit0 = unit0;
          break;
        }
        at += n * a.Hkv;
      }
    }
    return left > 0;
  };
  bool work = false;
  if (one_each) {
    if (sb0 < sb1) mine = seq_keys(a, sb0);
    work = form_share();
  }
  pdl_wait();
  pdl_trigger();
  bool again = !one_each;
  if (one_each) {
    const SeqKeys now = sb0 < sb1 ? seq_keys(a, sb0) : SeqKeys{0, 0};
    again = __syncthreads_or(now.L != mine.L || now.kbeg != mine.kbeg);  // (and the run is there for all)
    mine = now;
  }
  if (again) {
    work = form_share();
    __syncthreads();
  }
  // sequences that see no key, each written by a warp of one CTA
  for (int i = 0; i < per; ++i) {
    const int b = sb0 + i;
    bool empty = false;
    if (b < sb1 && b % nctas == cta) {
      const SeqKeys s = keys_of(b);
      empty = s.kbeg == s.L;
    }
    for (unsigned todo = __ballot_sync(0xffffffffu, empty); todo != 0; todo &= todo - 1) {
      const int eb = __shfl_sync(0xffffffffu, b, __ffs(todo) - 1);
      uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + static_cast<size_t>(eb) * a.H * HD);
      for (int x = lane; x < a.H * HD * C::ES / 16; x += 32) dst[x] = make_uint4(0, 0, 0, 0);
    }
  }
  if (!work) return;

  uint8_t* ring = smem + warp * (C::NST * 2 * C::STAGE_B);
  float* sc = sh.sc[warp];
  float* sa = sh.sa[warp];
  constexpr int kSh = 5 - ilog2(C::NP);
  const int hh = (lane >> kSh) & (G - 1);
  const float inv_cap = a.cap_log2 > 0.0f ? 1.0f / a.cap_log2 : 0.0f;
  int used = 0;  // stages that this warp has taken in earlier runs
  // After a wait that gave up (the error word is set) the CTA reads no further keys, but still takes its place in the
  // merges of this run and of those that follow, so that the counters are zero again for the next call.
  bool gave_up = false;

  while (true) {
    const Run run = sh.run;
    const size_t head_base = (static_cast<size_t>(run.b) * a.Hkv + run.kvh) * a.max_len;
    const T* gk = static_cast<const T*>(a.ck) + head_base * HD;
    const T* gv = static_cast<const T*>(a.cv) + head_base * HD;
    const int nstages = gave_up ? 0 : (run.k1 - run.k0 + C::SK - 1) / C::SK;
    auto issue = [&](int st_idx, int buf) {
      const int kk0 = run.k0 + st_idx * C::SK;
      const int n = min(C::SK, run.k1 - kk0);
      const uint32_t bytes = static_cast<uint32_t>(n) * C::ROWB;
      const uint32_t bar = smem_u32(&wbar[buf]);
      const uint32_t dk = smem_u32(ring + buf * 2 * C::STAGE_B);
      const uint32_t dv = dk + C::STAGE_B;
      mbar_arrive_expect_tx(bar, 2 * bytes);
      // (on a ring the rows wrap at most once: a run has at most max_len keys)
      const int r0 = a.ring ? kk0 % a.max_len : kk0;
      const int n0 = a.ring ? min(n, a.max_len - r0) : n;
      const uint32_t b0 = static_cast<uint32_t>(n0) * C::ROWB;
      bulk_g2s(dk, gk + static_cast<size_t>(r0) * HD, b0, bar);
      bulk_g2s(dv, gv + static_cast<size_t>(r0) * HD, b0, bar);
      if (n0 < n) {
        bulk_g2s(dk + b0, gk, bytes - b0, bar);
        bulk_g2s(dv + b0, gv, bytes - b0, bar);
      }
    };
    if (lane == 0) {
      for (int i = 0; i < C::NST; ++i) {
        const int st = warp + i * NW;
        if (st < nstages) issue(st, (used + i) % C::NST);
      }
    }

    // q of the G heads, pre-scaled into the log2 domain
    float2 q2[G][EL2], o2[G][EL2];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      float f[C::EL];
      load_row<T, C::NPC, C::PE>(static_cast<const T*>(a.q) + (static_cast<size_t>(run.b) * a.H + run.kvh * G + h) * HD, lane, f);
#pragma unroll
      for (int i = 0; i < C::EL; ++i) f[i] *= a.scale_log2;
      to_f2<C::EL>(f, q2[h]);
#pragma unroll
      for (int i = 0; i < EL2; ++i) o2[h][i] = make_float2(0.0f, 0.0f);
    }
    float m_l = -INFINITY, l_l = 0.0f;  // softmax state of head hh (log2 domain)
    const float slope = a.slopes != nullptr ? a.slopes[run.kvh * G + hh] * 1.4426950408889634f : 0.0f;

    bool aborted = false;
    int it = 0;
    for (;; ++it) {
      const int st_idx = warp + it * NW;
      if (st_idx >= nstages) break;
      const int buf = (used + it) % C::NST;
      if (!warp_wait(smem_u32(&wbar[buf]), ((used + it) / C::NST) & 1, a.err)) {
        aborted = true;
        break;
      }
      const int kk0 = run.k0 + st_idx * C::SK;
      const T* sk = reinterpret_cast<const T*>(ring + buf * 2 * C::STAGE_B);
      simt_stage<C, T, HD, G, true>(sk, sk + C::STAGE_B / C::ES, min(C::SK, run.k1 - kk0), q2, o2, m_l, l_l, sc, sa, lane,
                              [&](float s, int key) {
                                if (a.cap_log2 > 0.0f) s = a.cap_log2 * tanhf(s * inv_cap);
                                if (a.slopes != nullptr) s = fmaf(-slope, static_cast<float>(run.L - 1 - kk0 - key), s);
                                return s;
                              });
      __syncwarp();
      const int next = st_idx + C::NST * NW;
      if (lane == 0 && next < nstages) issue(next, buf);
    }
    // After a wait that gave up: wait (with a limit) for the copies that this warp still has in flight.
    if (aborted)
      for (int i = it; i < it + C::NST && warp + i * NW < nstages; ++i)
        warp_wait(smem_u32(&wbar[(used + i) % C::NST]), ((used + i) / C::NST) & 1, nullptr);
    used += it;
    if (__syncthreads_or(aborted)) gave_up = true;

    // ---- the warps' (m, l, o) meet in shared memory (the rings are free now)
    float* ms = reinterpret_cast<float*>(smem);  // [NW][G]
    float* ls = ms + NW * G;                     // [NW][G]
    float* os = ls + NW * G;                     // [NW][G][HD]
    if ((lane & ((1 << kSh) - 1)) == 0 && (lane >> kSh) < G) {
      ms[warp * G + hh] = m_l;
      ls[warp * G + hh] = l_l;
    }
#pragma unroll
    for (int h = 0; h < G; ++h) {
      float* orow = os + (warp * G + h) * HD;
#pragma unroll
      for (int c = 0; c < C::NPC; ++c) {
        float f[C::PE];
#pragma unroll
        for (int e = 0; e < C::PE; e += 2) {
          f[e] = o2[h][(c * C::PE + e) / 2].x;
          f[e + 1] = o2[h][(c * C::PE + e) / 2].y;
        }
        store_elems<C::PE>(orow + (lane + 32 * c) * C::PE, f);
      }
    }
    __syncthreads();
    const bool whole = run.nparts == 1;
    const int c_first = static_cast<int>(cta) - run.part;
    T* const out = static_cast<T*>(a.out) + (static_cast<size_t>(run.b) * a.H + run.kvh * G) * HD;
    const int slot = part_slot(c_first, run.part);
    for (int i4 = tid; i4 < G * HD / 4; i4 += NT) {
      const int h = i4 * 4 / HD, d = i4 * 4 % HD;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) M = fmaxf(M, ms[w * G + h]);
      float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float l = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float mw = ms[w * G + h];
        const float f = mw == -INFINITY ? 0.0f : ex2(mw - M);  // (a warp without a stage)
        const float4 v = *reinterpret_cast<const float4*>(os + (w * G + h) * HD + d);
        O.x = fmaf(f, v.x, O.x);
        O.y = fmaf(f, v.y, O.y);
        O.z = fmaf(f, v.z, O.z);
        O.w = fmaf(f, v.w, O.w);
        l = fmaf(f, ls[w * G + h], l);
      }
      if (whole) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const float f[4] = {O.x * inv, O.y * inv, O.z * inv, O.w * inv};
        store_elems<4>(out + i4 * 4, f);
      } else {
        *reinterpret_cast<float4*>(a.ws_o + static_cast<size_t>(slot) * G * HD + i4 * 4) = O;
        if (d == 0) a.ws_ml[slot * G + h] = make_float2(M, l);
      }
    }

    if (!whole) {
      // Parts are merged kFan neighbours at a time by the CTA that completes them,
      // each merge left in the slot of its first part, until one is left.
      int part = run.part, nleft = run.nparts, step = 1;
      unsigned* tickets = a.tickets;  // [level][slot of a merge's first part]
#pragma unroll 1
      while (true) {
        const int first = part / kFan * kFan, n = min(kFan, nleft - first);
        __threadfence();
        __syncthreads();
        if (tid == 0) {
          unsigned* ticket = tickets + part_slot(c_first, first * step);
          sh.last = atomicAdd(ticket, 1u) == static_cast<unsigned>(n - 1);
          if (sh.last) *ticket = 0u;  // ready for the next call
        }
        __syncthreads();
        if (!sh.last) break;
        __threadfence();
        const bool final = nleft <= kFan;
        const int first_slot = part_slot(c_first, first * step);
#pragma unroll 1
        for (int i4 = tid; i4 < G * HD / 4; i4 += NT) {
          const int h = i4 * 4 / HD;
          float2 ml[kFan];
          float4 v[kFan];
#pragma unroll
          for (int i = 0; i < kFan; ++i) {
            const int from = part_slot(c_first, (first + min(i, n - 1)) * step);
            ml[i] = __ldcg(&a.ws_ml[from * G + h]);
            v[i] = __ldcg(reinterpret_cast<const float4*>(a.ws_o + static_cast<size_t>(from) * G * HD) + i4);
          }
          float M = -INFINITY, l = 0.0f;
          float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < kFan; ++i) M = fmaxf(M, ml[i].x);
#pragma unroll
          for (int i = 0; i < kFan; ++i) {
            if (i < n) {
              const float f = ml[i].x == -INFINITY ? 0.0f : ex2(ml[i].x - M);
              l = fmaf(f, ml[i].y, l);
              O.x = fmaf(f, v[i].x, O.x);
              O.y = fmaf(f, v[i].y, O.y);
              O.z = fmaf(f, v[i].z, O.z);
              O.w = fmaf(f, v[i].w, O.w);
            }
          }
          if (final) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const float f[4] = {O.x * inv, O.y * inv, O.z * inv, O.w * inv};
            store_elems<4>(out + i4 * 4, f);
          } else {
            *reinterpret_cast<float4*>(a.ws_o + static_cast<size_t>(first_slot) * G * HD + i4 * 4) = O;
            if (i4 * 4 % HD == 0) {  // (written once every thread has read the first part's)
              sh.ml[0][h] = M;
              sh.ml[1][h] = l;
            }
          }
        }
        if (final) break;
        __syncthreads();
        if (tid < G) a.ws_ml[first_slot * G + tid] = make_float2(sh.ml[0][tid], sh.ml[1][tid]);
        part /= kFan;
        nleft = (nleft + kFan - 1) / kFan;
        step *= kFan;
        tickets += 2 * kMaxCtas;
      }
    }

    // ---- the share's next unit
    if (cut_units) return;
    left -= run.k1 - run.k0;
    if (left <= 0) return;
    fence_proxy_async_smem();  // (the next copies come after the stores to their place)
    __syncthreads();
    if (tid == 0) {
      int b = run.b, kvh = run.kvh + 1;
      SeqKeys s = seq_keys(a, b);
      long long unit0 = sh.unit0 + (s.L - s.kbeg);
      if (kvh == a.Hkv) {
        kvh = 0;
        do s = seq_keys(a, ++b);
        while (s.L == s.kbeg);  // (keys are left, so a sequence that has some follows)
      }
      const long long n = s.L - s.kbeg, c1 = (unit0 + n - 1) / share;
      sh.run = {b, kvh, s.kbeg, static_cast<int>(min(static_cast<long long>(s.L), s.kbeg + left)), s.L, 0,
                static_cast<int>(c1 - cta + 1)};
      sh.unit0 = unit0;
    }
    __syncthreads();
  }
}

template <typename T, int HD, int G, int NW>
cudaError_t launch_w(const ModsDecodeArgs& a, cudaStream_t s) {
  using C = SimtCfg<T, HD, G, NW, kBatch<HD * sizeof(T)>>;
  constexpr int smem = C::AREA_B + sizeof(Tail<NW, C::NST, G>);
  const cudaError_t e = set_smem_limit_once<decode_mods_kernel<T, HD, G, NW>>(smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.nctas));
  cfg.blockDim = dim3(NW * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_mods_kernel<T, HD, G, NW>, a);
}

template <typename T, int HD, int G>
cudaError_t launch_g(const ModsDecodeArgs& a, int warps, cudaStream_t s) {
  return warps == 8 ? launch_w<T, HD, G, 8>(a, s) : launch_w<T, HD, G, 4>(a, s);
}

template <typename T, int HD>
cudaError_t launch_h(const ModsDecodeArgs& a, int warps, cudaStream_t s) {
  switch (a.H / a.Hkv) {
    case 1: return launch_g<T, HD, 1>(a, warps, s);
    case 2: return launch_g<T, HD, 2>(a, warps, s);
    case 4: return launch_g<T, HD, 4>(a, warps, s);
    case 8:
      if constexpr (HD <= 256) return launch_g<T, HD, 8>(a, warps, s);
      return cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
}

template <typename T>
cudaError_t launch_t(const ModsDecodeArgs& a, int warps, cudaStream_t s) {
  switch (a.hd) {
    case 64: return launch_h<T, 64>(a, warps, s);
    case 128: return launch_h<T, 128>(a, warps, s);
    case 256: return launch_h<T, 256>(a, warps, s);
    case 512: return launch_h<T, 512>(a, warps, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_decode_mods(const ModsDecodeArgs& a, int dtype, int warps, cudaStream_t s) {
  return dtype == 1 ? launch_t<__nv_bfloat16>(a, warps, s) : launch_t<float>(a, warps, s);
}

ModsDecodePlan mods_decode_plan(int dtype, int window, int hd, int H, int Hkv, int B, int max_seq_len) {
  ModsDecodePlan p;
  const int span = window > 0 && window < max_seq_len ? window : max_seq_len;
  const int G = H / Hkv;
  const long long units = static_cast<long long>(B) * Hkv;
  p.win = units <= 0x7fffffffLL && decode_win_eligible(dtype, hd, G, span, static_cast<int>(units));
  if (p.win) {
    p.nctas = p.warps = 0;
    p.t_bytes = p.ml_bytes = p.o_bytes = p.ws_bytes = 0;
    return p;
  }
  const long long most = units * ((static_cast<long long>(span) + kMinShare - 1) / kMinShare);  // CTAs with a share
  // One CTA of 8 warps per SM where there is no more than that to do; and for rows of 1 KB or more with few units, whose
  // parts are then half as many to merge (head_dim 512, 1 x 20000 keys 25.6 us against 30.3 with two of 4 warps, 32 x 1000
  // .. 8000 105 against 110; float32, head_dim 256, 32 x 1024 .. 4096 59 against 72).  Narrow rows, many units, or long
  // shares, which two CTAs per SM stream better: 4 warps (64 x 1024 .. 8192 of head_dim 128 92 us against 104, 64 x 100
  // .. 2000 of 512 62 against 64, 4 x 131072 of 512 250 against 263).
  const bool wide = hd * (dtype == 1 ? 2 : 4) >= 1024 && 2 * units <= sm_count() && units * span <= 4096LL * sm_count();
  p.warps = most <= sm_count() || wide ? 8 : 4;
  // (few units have more parts to merge then: 1 x 30000 keys of head_dim 128 17.7 us with four CTAs per SM, 16.0 with three)
  const int resident = std::min(units < 32 ? 3 : 4, resident_ctas(p.warps, G * hd, hd * (dtype == 1 ? 2 : 4)));
  const long long slots = static_cast<long long>(sm_count()) * resident;
  p.nctas = static_cast<int>(most < slots ? most : slots);
  if (p.nctas > kMaxCtas) p.nctas = kMaxCtas;
  const size_t n = static_cast<size_t>(p.nctas);
  p.t_bytes = kTicketBytes;
  p.ml_bytes = (2 * n * G * sizeof(float2) + 255) / 256 * 256;
  p.o_bytes = (2 * n * G * hd * sizeof(float) + 255) / 256 * 256;
  p.ws_bytes = p.nctas > 1 ? p.t_bytes + p.ml_bytes + p.o_bytes : 0;
  return p;
}

}  // namespace g4
