// The paged 4-bit KV cache: block tables and slots from request lengths, and
// the read-back to bf16.  (The append: g4_append.cu.)
// Formats and byte order: include/g4attn.h, g4_kv4.cuh.
#include <cooperative_groups.h>

#include "g4_device.cuh"
#include "g4_kv4_internal.h"
#include "g4_kv4.cuh"

namespace g4 {
namespace {

namespace cg = cooperative_groups;

template <typename Args>
cudaError_t launch_pdl(void (*kern)(Args), dim3 grid, unsigned block, size_t smem, unsigned cluster, cudaStream_t s,
                       const Args& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

// ---------------------------------------------------------------- block assignment
//
// need_b = max(0, ceil(new_b / bs) - ceil(old_b / bs)) blocks are taken and
// ret_b = max(0, ceil(old_b / bs) - ceil(new_b / bs)) given back; their
// exclusive prefix sums over b give each sequence its place in the free list,
// so the result does not depend on the order in which threads run.
//
// One cluster.  Every CTA scans all B lengths (both sums packed in one 64-bit
// word; a few KB from L2, cheaper than exchanging partial sums) and keeps the sums
// in shared memory, then serves its own share of the sequences: it pushes their
// returned blocks, waits for the cluster (blocks given back may be taken in the
// same call), pops, and writes lengths, positions and slots.  Pushes and pops are
// dealt out one block per thread, its sequence found in the sums by bisection.
// The sums take every entry given back for a block.  Where one is no block of the
// pool (a caller may have taken it away), the threads that meet such entries tell
// all CTAs how many, and after the barrier the pushes are made again without
// them, behind another barrier; where there are none this costs nothing but a
// reduction over the warp.
//   Bound by latency: lengths, free list and table are dependent reads, with
// one cluster barrier between them; with many new tokens also by the
// instructions that form positions and slots.  Measured: 64 sequences of a token
// each 4.3 us (the host's call takes 5.4); 96 sequences of up to 2048 tokens (1.6 MB
// of positions and slots) 6.6 us with a cluster of 16, 8.5 with 8, 12.5 with 4; rows of
// 2047 tokens, which are not written four at a time, 7.4.

// (512: 12.0 us against 9.3 in that case, when the largest cluster had 8 CTAs.)
constexpr int kAssignThreads = 1024;
constexpr int kAssignMaxCtas = 16;

// The first i in [lo, hi) with v[i] > x (hi if there is none); v ascends.
__device__ __forceinline__ int first_above(const int* v, int lo, int hi, int x) {
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kAssignThreads) kv4_assign_kernel(const __grid_constant__ Kv4AssignArgs a) {
  extern __shared__ int s_mem[];
  __shared__ unsigned long long s_warp[kAssignThreads / 32];
  __shared__ int s_gone[kAssignMaxCtas];  // entries without a block among those that CTA r gives back
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NW = kAssignThreads / 32;
  const int nctas = gridDim.x, rank = blockIdx.x;
  const int per = (a.B + nctas - 1) / nctas;
  const int b0 = min(a.B, rank * per), b1 = min(a.B, b0 + per);  // this CTA's sequences
  int* taken = s_mem;           // [B] blocks taken up to and including b
  int* given = taken + a.B;     // [B] blocks given back up to and including b
  int* s_old = given + a.B;     // [per] lengths of its sequences, clamped to the contract
  int* s_new = s_old + per;
  const long long most = static_cast<long long>(a.max_blocks) << a.block_shift;
  const int cap = static_cast<int>(most > 0x7fffffffLL ? 0x7fffffffLL : most);
  const int mask = (1 << a.block_shift) - 1;
  auto blocks_of = [&](int len) { return (len >> a.block_shift) + ((len & mask) != 0); };

  if (tid < kAssignMaxCtas) s_gone[tid] = 0;
  if (nctas > 1) cluster.barrier_arrive();  // (others may add to s_gone past the wait below)
  pdl_wait();
  pdl_trigger();
  const int count = min(max(__ldcg(a.free_count), 0), a.n_blocks);
  unsigned long long carry = 0;
  for (int base = 0; base < a.B; base += kAssignThreads) {
    const int b = base + tid;
    unsigned long long v = 0;
    if (b < a.B) {
      const int was = min(max(__ldcg(a.old_lens + b), 0), cap);
      int len = min(max(__ldcg(a.new_lens + b), 0), cap);
      if (len - was > a.T) len = was + a.T;  // (both in [0, 2^31): no overflow)
      if (b >= b0 && b < b1) {
        s_old[b - b0] = was;
        s_new[b - b0] = len;
      }
      const int d = blocks_of(len) - blocks_of(was);
      v = d >= 0 ? static_cast<unsigned>(d) : static_cast<unsigned long long>(static_cast<unsigned>(-d)) << 32;
    }
    unsigned long long sum = v;  // inclusive over the warp; neither half can carry (B * max_blocks < 2^31)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    unsigned long long all = lane < NW ? s_warp[lane] : 0;  // every warp scans the warps' sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long u = __shfl_up_sync(0xffffffffu, all, o);
      if (lane >= o) all += u;
    }
    const unsigned long long before = __shfl_sync(0xffffffffu, all, warp == 0 ? 0 : warp - 1);
    sum += carry + (warp == 0 ? 0 : before);
    if (b < a.B) {
      taken[b] = static_cast<int>(sum & 0xffffffffu);
      given[b] = static_cast<int>(sum >> 32);
    }
    carry += __shfl_sync(0xffffffffu, all, 31);
    __syncthreads();
  }
  const int back = static_cast<int>(carry >> 32);
  if (nctas > 1) cluster.barrier_wait();

  // Blocks given back by this CTA's sequences: the x-th of the call goes behind
  // the free list's first `count`.
  const int g0 = b0 > 0 ? given[b0 - 1] : 0, g1 = b1 > b0 ? given[b1 - 1] : g0;
  auto given_id = [&](int x) {
    const int b = first_above(given, b0, b1, x);
    const int e = blocks_of(s_new[b - b0]) + x - (b > 0 ? given[b - 1] : 0);
    return __ldcg(a.table + static_cast<size_t>(b) * a.max_blocks + e);
  };
  auto in_pool = [&](int id) { return id >= 0 && id < a.n_blocks; };
  auto push = [&](long long at, int id) {
    if (at < a.n_blocks) a.free_blocks[at] = id;
  };
  auto sync_all = [&] {
    if (nctas > 1) {
      cluster.sync();
    } else {
      __syncthreads();
    }
  };
  int gone = 0;
  for (int x = g0 + tid; x < g1; x += kAssignThreads) {
    const int id = given_id(x);
    if (in_pool(id))
      push(static_cast<long long>(count) + x, id);
    else
      ++gone;
  }
  gone = __reduce_add_sync(0xffffffffu, gone);
  if (gone != 0 && lane < nctas) atomicAdd(nctas > 1 ? cluster.map_shared_rank(&s_gone[rank], lane) : &s_gone[0], gone);
  // Blocks given back are in place, and every CTA has read the lengths and the
  // count, which the outputs may overwrite.
  sync_all();
  int gone_all = 0;
  const int gone_of = lane < nctas ? s_gone[lane] : 0;
  if (__any_sync(0xffffffffu, gone_of != 0)) {  // (the same for all CTAs)
    gone_all = __reduce_add_sync(0xffffffffu, gone_of);
    const int gone_before = __reduce_add_sync(0xffffffffu, lane < rank ? gone_of : 0);
    long long at = static_cast<long long>(count) + g0 - gone_before;
    for (int x0 = g0; x0 < g1; x0 += kAssignThreads) {
      const int x = x0 + tid;
      const int id = x < g1 ? given_id(x) : -1;
      const unsigned votes = __ballot_sync(0xffffffffu, in_pool(id));
      if (lane == 0) s_warp[warp] = __popc(votes);
      __syncthreads();
      int before = 0, all = 0;  // in the warps before this one; in all
      for (int w = 0; w < NW; ++w) {
        const int n = static_cast<int>(s_warp[w]);
        if (w < warp) before += n;
        all += n;
      }
      if (in_pool(id)) push(at + before + __popc(votes & ((1u << lane) - 1)), id);
      at += all;
      __syncthreads();
    }
    sync_all();
  }
  const int there =
      static_cast<int>(min(static_cast<long long>(count) + back - gone_all, static_cast<long long>(a.n_blocks)));
  // Blocks taken: the x-th of the call is the free list's x-th from its top.  A
  // sequence is served if the blocks of all up to it are there.
  const int t0 = b0 > 0 ? taken[b0 - 1] : 0, t1 = b1 > b0 ? min(taken[b1 - 1], there) : t0;
  for (int x = t0 + tid; x < t1; x += kAssignThreads) {
    const int b = first_above(taken, b0, b1, x);
    if (taken[b] <= there)
      a.table[static_cast<size_t>(b) * a.max_blocks + blocks_of(s_old[b - b0]) + x - (b > 0 ? taken[b - 1] : 0)] =
          __ldcg(a.free_blocks + (there - 1 - x));
  }
  __syncthreads();
  // granted lengths (a sequence that needs no blocks is always served)
  for (int i = tid; i < b1 - b0; i += kAssignThreads) {
    const int b = b0 + i;
    const bool needs = taken[b] > (b > 0 ? taken[b - 1] : 0);
    const int len = needs && taken[b] > there ? s_old[i] : s_new[i];
    s_new[i] = len;
    a.lens_out[b] = len;
  }
  // The served ones are those up to some sequence, whose sum is what was taken.
  if (rank == 0) {
    if (tid == 0 && (a.B == 0 || taken[0] > there)) *a.count_out = there;
    for (int b = tid; b < a.B; b += kAssignThreads)
      if (taken[b] <= there && (b + 1 == a.B || taken[b + 1] > there)) *a.count_out = there - taken[b];
  }
  __syncthreads();

  // positions and slots, four neighbours of a row (in at most two blocks) per
  // thread where rows allow it
  const int nb = b1 - b0;
  // What is added to a position of table entry e to get its slot, and what is or-ed to the sum (-1: an id outside the pool).
  auto slot_base = [&](int id, int e, int& none) {
    none = id >= 0 && id < a.n_blocks ? 0 : -1;
    return static_cast<int>(static_cast<unsigned>(id - e) << a.block_shift);
  };
  if ((a.T & 3) == 0 && ((reinterpret_cast<uintptr_t>(a.positions) | reinterpret_cast<uintptr_t>(a.slots)) & 15) == 0) {
    const unsigned quads = static_cast<unsigned>(a.T) / 4, n = static_cast<unsigned>(nb) * quads;
    const unsigned dr = quads > 0 ? kAssignThreads / quads : 0, dt = kAssignThreads - dr * quads;
    unsigned r = quads > 0 ? tid / quads : 0, t = tid - r * quads;  // row and quad of i
    int4* const pos4 = reinterpret_cast<int4*>(a.positions) + static_cast<size_t>(b0) * quads;
    int4* const slot4 = reinterpret_cast<int4*>(a.slots) + static_cast<size_t>(b0) * quads;
#pragma unroll 2
    for (unsigned i = tid; i < n; i += kAssignThreads) {
      const unsigned at = static_cast<unsigned>(s_old[r]) + 4 * t, end = static_cast<unsigned>(s_new[r]);  // (at < 2^32)
      int p[4] = {-1, -1, -1, -1}, q[4] = {-1, -1, -1, -1};
      if (at < end) {
        const int32_t* row = a.table + static_cast<size_t>(b0 + static_cast<int>(r)) * a.max_blocks;
        const int e = static_cast<int>(at >> a.block_shift);
        const unsigned next = static_cast<unsigned>(e + 1) << a.block_shift;  // first position of the next block
        int none0, none1, base0 = slot_base(row[e], e, none0), base1 = base0;
        none1 = none0;
        if (next < min(at + 4, end)) base1 = slot_base(row[e + 1], e + 1, none1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const unsigned pos = at + k;
          if (pos < end) {
            p[k] = static_cast<int>(pos);
            q[k] = (static_cast<int>(pos) + (pos < next ? base0 : base1)) | (pos < next ? none0 : none1);
          }
        }
      }
      pos4[i] = make_int4(p[0], p[1], p[2], p[3]);
      slot4[i] = make_int4(q[0], q[1], q[2], q[3]);
      r += dr;
      t += dt;
      if (t >= quads) {
        t -= quads;
        ++r;
      }
    }
  } else if (a.T > 0) {
    const unsigned T = static_cast<unsigned>(a.T), n = static_cast<unsigned>(nb) * T;
    const unsigned dr = kAssignThreads / T, dt = kAssignThreads - dr * T;
    unsigned r = tid / T, t = tid - r * T;
    int32_t* const pos1 = a.positions + static_cast<size_t>(b0) * T;
    int32_t* const slot1 = a.slots + static_cast<size_t>(b0) * T;
#pragma unroll 4
    for (unsigned i = tid; i < n; i += kAssignThreads) {
      const unsigned at = static_cast<unsigned>(s_old[r]) + t;
      int pos = -1, slot = -1;
      if (at < static_cast<unsigned>(s_new[r])) {
        const int e = static_cast<int>(at >> a.block_shift);
        int none;
        slot = slot_base(a.table[static_cast<size_t>(b0 + static_cast<int>(r)) * a.max_blocks + e], e, none);
        pos = static_cast<int>(at);
        slot = (slot + pos) | none;
      }
      pos1[i] = pos;
      slot1[i] = slot;
      r += dr;
      t += dt;
      if (t >= T) {
        t -= T;
        ++r;
      }
    }
  }
}

// ---------------------------------------------------------------- gather
//
// A warp per 64-element piece of a record: 16-byte loads in fragment order,
// values as fp16 code times scale (exact), written as bf16; a K store writes 8
// bytes per lane (32 contiguous per row), a V store 4.  One piece per warp keeps
// a small gather (a step's new rows) to one round of loads.
//   Bound by its writes, 3.6 times what it reads.  Measured at head_dim 512, 2 kv
// heads: 8 sequences of 4096 rows (268 MB written) 26.7 us, where the bytes alone
// take 24 at the rate of a copy (a part of them stays in L2); one of 700 rows 2.9
// us.  (A warp for a whole record, its pieces one after another: 34.8 and 4.0 us.)

// Most CTAs of a launch, which take turns beyond that.  A prefill's rows are
// bounded on the host and counted on the device: 4 sequences of 2000 keys and 256
// new tokens (head_dim 512) under a bound of 131072 take 63.5 us against 119.6 with
// a CTA for every 16 rows of the bound, 61 under one of 4096.  9728 CTAs: 66.2; 2736:
// 62.0, but 8 sequences of 4096 rows 28.3 us against 26.9.
constexpr int kGatherCtas = 4864;

template <int HD>
__global__ void __launch_bounds__(256) kv4_gather_kernel(const __grid_constant__ Kv4GatherArgs a) {
  using R = Kv4Rec<HD>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int p = (threadIdx.x >> 5) % R::NP;
  const int unit = blockIdx.x / a.per_unit;
  constexpr int kPerCta = 8 / R::NP;  // records
  pdl_wait();
  pdl_trigger();
  const int b = unit / a.Hkv, kvh = unit % a.Hkv;
  int gi = blockIdx.x % a.per_unit * kPerCta + (threadIdx.x >> 5) / R::NP;

  long long first;
  int rows = a.rows;
  if (a.q_start != nullptr) {
    const int q0 = min(max(a.q_start[b], 0), a.max_seq_len);
    const int low = a.window > 0 ? max(0, q0 - a.window + 1) : 0;
    if (gi == 0 && kvh == 0 && p == 0 && lane == 0) a.q_rel[b] = q0 - low;
    first = low;
    rows = min(rows, q0 - low + a.T);
  } else {
    first = a.start[b];
  }
  const int len = a.lens[b];
  __nv_bfloat16* ko = static_cast<__nv_bfloat16*>(a.k) + static_cast<size_t>(unit) * a.rows * HD;
  __nv_bfloat16* vo = static_cast<__nv_bfloat16*>(a.v) + static_cast<size_t>(unit) * a.rows * HD;

#pragma unroll 1
  for (;; gi += a.per_unit * kPerCta) {
    // group numbers round towards minus infinity, so a group never straddles position 0
    const long long pos0 = ((first >> 4) + gi) << 4;
    if (pos0 >= first + rows) return;
    const int entry = pos0 >= 0 ? static_cast<int>(pos0 >> a.block_shift) : -1;
    int block = -1;
    if (pos0 >= 0 && pos0 < len && entry < a.max_blocks) block = a.table[static_cast<size_t>(b) * a.max_blocks + entry];
    const bool there = block >= 0 && block < a.n_blocks;
    const int in_block = static_cast<int>(pos0 & ((1 << a.block_shift) - 1));
    const uint8_t* rec = there ? a.data + kv4_record<HD>(block, kvh, in_block >> 4, a.Hkv, a.block_shift) : nullptr;

    // Of the record's 16 positions: the row of the first, and how many are held.
    const int row0 = static_cast<int>(pos0 - first);
    const int nheld = there ? static_cast<int>(min(16LL, len - pos0)) : 0;

    // fp16x2 code times scale, then the exponent, as bf16x2
    auto value = [](uint32_t codes, __half2 s, float mul) -> uint32_t {
      const float2 v = __half22float2(__hmul2(as_half2(codes), s));
      return pack_bf16x2(v.x * mul, v.y * mul);
    };
    uint4 kc = make_uint4(0, 0, 0, 0), vc = kc, vs = kc;
    uint2 ks = make_uint2(0, 0);
    if (there) {
      kc = *reinterpret_cast<const uint4*>(rec + R::KC + p * 512 + lane * 16);
      ks = *reinterpret_cast<const uint2*>(rec + R::KS + p * 64 + g * 8);
      vc = *reinterpret_cast<const uint4*>(rec + R::VC + p * 512 + lane * 16);
      vs = *reinterpret_cast<const uint4*>(rec + R::VS + p * 64 + t * 16);
    }
    const uint32_t kw[2][2] = {{kc.x, kc.y}, {kc.z, kc.w}};
    const uint32_t vw[4] = {vc.x, vc.y, vc.z, vc.w};
    const uint32_t vsw[4] = {vs.x, vs.y, vs.z, vs.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const __half2 s = as_half2(w & 1 ? e4m3x2_hi_f16x2(w < 2 ? ks.x : ks.y) : e4m3x2_f16x2(w < 2 ? ks.x : ks.y));
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int m = 8 * r + g;
        if (static_cast<unsigned>(row0 + m) < static_cast<unsigned>(rows)) {
          const __half2 sr = r == 0 ? __low2half2(s) : __high2half2(s);
          uint2 o = make_uint2(0, 0);
          if (m < nheld) {
            const uint32_t word = kw[r][w >> 1];
            o.x = value(w & 1 ? e2m1x2_f16x2<2>(word) : e2m1x2_f16x2<0>(word), sr, a.k_mul);
            o.y = value(w & 1 ? e2m1x2_f16x2<3>(word) : e2m1x2_f16x2<1>(word), sr, a.k_mul);
          }
          *reinterpret_cast<uint2*>(ko + static_cast<size_t>(row0 + m) * HD + p * 64 + w * 16 + t * 4) = o;
        }
      }
      const __half2 s01 = as_half2(e4m3x2_f16x2(vsw[w])), s23 = as_half2(e4m3x2_hi_f16x2(vsw[w]));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = 8 * (i >> 1) + 2 * t + (i & 1);
        if (static_cast<unsigned>(row0 + m) < static_cast<unsigned>(rows)) {
          const __half2 sp = i < 2 ? s01 : s23;
          const __half2 si = i & 1 ? __high2half2(sp) : __low2half2(sp);
          uint32_t codes;
          switch (w) {
            case 0: codes = e2m1x2_f16x2<0>(vw[i]); break;
            case 1: codes = e2m1x2_f16x2<1>(vw[i]); break;
            case 2: codes = e2m1x2_f16x2<2>(vw[i]); break;
            default: codes = e2m1x2_f16x2<3>(vw[i]); break;
          }
          *reinterpret_cast<uint32_t*>(vo + static_cast<size_t>(row0 + m) * HD + p * 64 + w * 16 + g * 2) =
              m < nheld ? value(codes, si, 1.0f) : 0u;
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv4_assign(const Kv4AssignArgs& a, cudaStream_t s) {
  // A CTA per 4096 positions (2048 or 8192: the same within 1 %) or 64 sequences
  // (1000 that gain a token or end: 5.0 us against 11.3 with one CTA, 6.6 with one per
  // 256; one per 32 makes 64 of them 4.5 against 4.2), up to 16 (the largest cluster,
  // where one of them fits the device; 8 are always allowed).
  const cudaError_t e = set_smem_limit_once<kv4_assign_kernel>(kKv4MaxBatch * 16);
  if (e != cudaSuccess) return e;
  constexpr size_t kMostSmem = (2 * kKv4MaxBatch + 2 * (kKv4MaxBatch / kAssignMaxCtas)) * 4;  // of a CTA of 16
  const unsigned most = cluster_limit_once<kv4_assign_kernel>(kAssignThreads, kMostSmem);
  const long long work = static_cast<long long>(a.B) * a.T;
  unsigned n = 1;
  while (n < most && n < static_cast<unsigned>(a.B) && (work > 4096LL * n || a.B > 64 * static_cast<int>(n))) n *= 2;
  const size_t per = (static_cast<size_t>(a.B) + n - 1) / n;
  const size_t smem = (2 * static_cast<size_t>(a.B) + 2 * per) * 4;
  return launch_pdl(kv4_assign_kernel, dim3(n), kAssignThreads, smem, n, s, a);
}

cudaError_t launch_kv4_gather(const Kv4GatherArgs& args, cudaStream_t s) {
  const long long units = static_cast<long long>(args.B) * args.Hkv;
  if (units > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int per = 8 * 64 / args.hd;                            // records per CTA of 8 warps
  const int need = (args.rows / kKv4Group + 2 + per - 1) / per;  // CTAs for the groups that rows positions can touch
  const long long room = kGatherCtas / units;
  Kv4GatherArgs a = args;
  a.per_unit = need < room ? need : room > 0 ? static_cast<int>(room) : 1;
  const dim3 grid(static_cast<unsigned>(units * a.per_unit));
  switch (a.hd) {
    case 64: return launch_pdl(kv4_gather_kernel<64>, grid, 256, 0, 1, s, a);
    case 128: return launch_pdl(kv4_gather_kernel<128>, grid, 256, 0, 1, s, a);
    case 256: return launch_pdl(kv4_gather_kernel<256>, grid, 256, 0, 1, s, a);
    case 512: return launch_pdl(kv4_gather_kernel<512>, grid, 256, 0, 1, s, a);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace g4
