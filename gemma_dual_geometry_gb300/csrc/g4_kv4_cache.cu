// The paged 4-bit KV cache: block tables and slots from request lengths, and
// the read-back to bf16.  (The append: g4_append.cu.)
// Formats and byte order: include/g4attn.h, g4_kv4.cuh.
#include <cooperative_groups.h>

#include "g4_device.cuh"
#include "g4_internal.h"
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
// word; a few KB from L2, cheaper than exchanging partial sums), then serves
// its own share of the sequences: it pushes their returned blocks, waits for
// the cluster (blocks given back may be taken in the same call), pops, and
// writes the positions and slots.  Bound by latency: three dependent global
// reads (lengths, free list, table) and one cluster barrier.

constexpr int kAssignThreads = 512;

// Block lengths of one sequence, clamped to the contract.
struct Span {
  int old_len, new_len, have, want;
};
__device__ __forceinline__ Span span_of(const Kv4AssignArgs& a, int b) {
  const long long most = static_cast<long long>(a.max_blocks) << a.block_shift;
  const int cap = static_cast<int>(most > 0x7fffffffLL ? 0x7fffffffLL : most);
  Span s;
  s.old_len = min(max(__ldcg(a.old_lens + b), 0), cap);
  const long long grown = static_cast<long long>(s.old_len) + a.T;
  s.new_len = min(max(__ldcg(a.new_lens + b), 0), cap);
  if (s.new_len > grown) s.new_len = static_cast<int>(grown);
  // (the sum in 64 bits: a length may be within a block of 2^31)
  const long long up = (1 << a.block_shift) - 1;
  s.have = static_cast<int>((s.old_len + up) >> a.block_shift);
  s.want = static_cast<int>((s.new_len + up) >> a.block_shift);
  return s;
}

__global__ void __launch_bounds__(kAssignThreads) kv4_assign_kernel(const __grid_constant__ Kv4AssignArgs a) {
  extern __shared__ int s_sums[];  // [B] blocks taken up to and including b; [B] given back before b
  __shared__ unsigned long long s_warp[kAssignThreads / 32];
  __shared__ unsigned long long s_carry;
  __shared__ int s_taken;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NW = kAssignThreads / 32;
  const int nctas = gridDim.x, rank = blockIdx.x;
  int* upto = s_sums;
  int* before = s_sums + a.B;

  pdl_wait();
  pdl_trigger();
  const int count = min(max(__ldcg(a.free_count), 0), a.n_blocks);
  unsigned long long carry = 0;
  for (int base = 0; base < a.B; base += kAssignThreads) {
    const int b = base + tid;
    unsigned long long v = 0;
    if (b < a.B) {
      const Span s = span_of(a, b);
      v = static_cast<unsigned long long>(static_cast<unsigned>(max(s.have - s.want, 0))) << 32 |
          static_cast<unsigned>(max(s.want - s.have, 0));
    }
    unsigned long long sum = v;  // inclusive over the warp; neither half can carry (B * max_blocks < 2^31)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    unsigned long long pre = carry;
    for (int w = 0; w < warp; ++w) pre += s_warp[w];
    sum += pre;
    if (b < a.B) {
      upto[b] = static_cast<int>(sum & 0xffffffffu);
      before[b] = static_cast<int>((sum - v) >> 32);
    }
    if (tid == kAssignThreads - 1) s_carry = sum;
    __syncthreads();
    carry = s_carry;
  }
  if (tid == 0) s_taken = 0;
  const int there = static_cast<int>(min(static_cast<long long>(count) + static_cast<long long>(carry >> 32),
                                         static_cast<long long>(a.n_blocks)));

  // this CTA's sequences
  const int per = (a.B + nctas - 1) / nctas;
  const int b0 = min(a.B, rank * per), b1 = min(a.B, b0 + per);
  for (int b = b0 + warp; b < b1; b += NW) {
    const Span s = span_of(a, b);
    for (int e = s.want + lane; e < s.have; e += 32) {
      const long long at = static_cast<long long>(count) + before[b] + (e - s.want);
      if (at < a.n_blocks) a.free_blocks[at] = __ldcg(a.table + static_cast<size_t>(b) * a.max_blocks + e);
    }
  }
  // Blocks given back are in place (and every CTA has read the lengths and the
  // count, which the outputs may overwrite).
  if (nctas > 1) {
    cluster.sync();
  } else {
    __syncthreads();
  }
  for (int b = b0 + warp; b < b1; b += NW) {
    const Span s = span_of(a, b);
    const int need = s.want - s.have;
    if (need > 0 && upto[b] <= there) {
      const int top = there - 1 - (upto[b] - need);
      for (int j = lane; j < need; j += 32)
        a.table[static_cast<size_t>(b) * a.max_blocks + s.have + j] = __ldcg(a.free_blocks + top - j);
    }
  }
  // Sequences that need blocks are granted in order, so the largest granted
  // prefix is what was taken; the first CTA forms it over all of them.
  if (rank == 0) {
    int taken = 0;
    for (int b = tid; b < a.B; b += kAssignThreads) {
      if (upto[b] <= there) taken = max(taken, upto[b]);
    }
    atomicMax(&s_taken, taken);
  }
  __syncthreads();
  if (rank == 0 && tid == 0) *a.count_out = there - s_taken;

  // positions and slots of its sequences, then their lengths
  const int block_mask = (1 << a.block_shift) - 1;
  const long long n = static_cast<long long>(b1 - b0) * a.T;
  for (long long i = tid; i < n; i += kAssignThreads) {
    const int q = static_cast<int>(static_cast<unsigned>(i) / static_cast<unsigned>(a.T));
    const int b = b0 + q, t = static_cast<int>(i - static_cast<long long>(q) * a.T);
    const Span s = span_of(a, b);
    const bool granted = s.want <= s.have || upto[b] <= there;
    const long long at = static_cast<long long>(s.old_len) + t;
    int pos = -1, slot = -1;
    if (granted && at < s.new_len) {
      pos = static_cast<int>(at);
      const int id = a.table[static_cast<size_t>(b) * a.max_blocks + (pos >> a.block_shift)];
      if (id >= 0 && id < a.n_blocks) slot = (id << a.block_shift) + (pos & block_mask);
    }
    const size_t o = static_cast<size_t>(b) * a.T + t;
    a.positions[o] = pos;
    a.slots[o] = slot;
  }
  __syncthreads();
  for (int b = b0 + tid; b < b1; b += kAssignThreads) {
    const Span s = span_of(a, b);
    a.lens_out[b] = s.want <= s.have || upto[b] <= there ? s.new_len : s.old_len;
  }
}

// ---------------------------------------------------------------- gather
//
// A warp per record: 16-byte loads in fragment order, values as fp16 code
// times scale (exact), written as bf16; a K store writes 8 bytes per lane (32
// contiguous per row), a V store 4.

template <int HD>
__global__ void __launch_bounds__(256) kv4_gather_kernel(const __grid_constant__ Kv4GatherArgs a) {
  using R = Kv4Rec<HD>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int ngroups = a.rows / kKv4Group + 2;  // that rows positions can touch
  const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const long long unit = item / ngroups;
  pdl_wait();
  pdl_trigger();
  if (unit >= static_cast<long long>(a.B) * a.Hkv) return;
  const int gi = static_cast<int>(item - unit * ngroups);
  const int b = static_cast<int>(unit / a.Hkv), kvh = static_cast<int>(unit % a.Hkv);

  long long first;
  int rows = a.rows;
  if (a.q_start != nullptr) {
    const int q0 = min(max(a.q_start[b], 0), a.max_seq_len - a.T);
    const int low = a.window > 0 ? max(0, q0 - a.window + 1) : 0;
    if (gi == 0 && kvh == 0 && lane == 0) a.q_rel[b] = q0 - low;
    first = low;
    rows = min(rows, q0 - low + a.T);
  } else {
    first = a.start[b];
  }
  // group numbers round towards minus infinity, so a group never straddles position 0
  const long long pos0 = ((first >> 4) + gi) << 4;
  if (pos0 >= first + rows) return;
  const int len = a.lens[b];
  const int entry = pos0 >= 0 ? static_cast<int>(pos0 >> a.block_shift) : -1;
  int block = -1;
  if (pos0 >= 0 && pos0 < len && entry < a.max_blocks) block = a.table[static_cast<size_t>(b) * a.max_blocks + entry];
  const bool there = block >= 0 && block < a.n_blocks;
  const int in_block = static_cast<int>(pos0 & ((1 << a.block_shift) - 1));
  const uint8_t* rec = there ? a.data + kv4_record<HD>(block, kvh, in_block >> 4, a.Hkv, a.block_shift) : nullptr;
  __nv_bfloat16* ko = static_cast<__nv_bfloat16*>(a.k) + static_cast<size_t>(unit) * a.rows * HD;
  __nv_bfloat16* vo = static_cast<__nv_bfloat16*>(a.v) + static_cast<size_t>(unit) * a.rows * HD;

  // fp16x2 code times scale, then the exponent, as bf16x2
  auto value = [](uint32_t codes, __half2 s, float mul) -> uint32_t {
    const float2 v = __half22float2(__hmul2(as_half2(codes), s));
    return pack_bf16x2(v.x * mul, v.y * mul);
  };
#pragma unroll
  for (int p = 0; p < R::NP; ++p) {
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
        const long long pos = pos0 + 8 * r + g;
        if (pos >= first && pos < first + rows) {
          const bool held = there && pos < len;
          const __half2 sr = r == 0 ? __low2half2(s) : __high2half2(s);
          uint2 o = make_uint2(0, 0);
          if (held) {
            const uint32_t word = kw[r][w >> 1];
            o.x = value(w & 1 ? e2m1x2_f16x2<2>(word) : e2m1x2_f16x2<0>(word), sr, a.k_mul);
            o.y = value(w & 1 ? e2m1x2_f16x2<3>(word) : e2m1x2_f16x2<1>(word), sr, a.k_mul);
          }
          *reinterpret_cast<uint2*>(ko + static_cast<size_t>(pos - first) * HD + p * 64 + w * 16 + t * 4) = o;
        }
      }
      const __half2 s01 = as_half2(e4m3x2_f16x2(vsw[w])), s23 = as_half2(e4m3x2_hi_f16x2(vsw[w]));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long pos = pos0 + 8 * (i >> 1) + 2 * t + (i & 1);
        if (pos >= first && pos < first + rows) {
          const bool held = there && pos < len;
          const __half2 sp = i < 2 ? s01 : s23;
          const __half2 si = i & 1 ? __high2half2(sp) : __low2half2(sp);
          uint32_t codes;
          switch (w) {
            case 0: codes = e2m1x2_f16x2<0>(vw[i]); break;
            case 1: codes = e2m1x2_f16x2<1>(vw[i]); break;
            case 2: codes = e2m1x2_f16x2<2>(vw[i]); break;
            default: codes = e2m1x2_f16x2<3>(vw[i]); break;
          }
          *reinterpret_cast<uint32_t*>(vo + static_cast<size_t>(pos - first) * HD + p * 64 + w * 16 + g * 2) =
              held ? value(codes, si, 1.0f) : 0u;
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv4_assign(const Kv4AssignArgs& a, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(a.B) * 8;
  if (smem > 40 * 1024) {
    const cudaError_t e = set_smem_limit_once<kv4_assign_kernel>(kKv4MaxBatch * 8);
    if (e != cudaSuccess) return e;
  }
  // Positions and slots are what grows: a CTA per 4096 of them, up to the portable cluster size.
  const long long work = static_cast<long long>(a.B) * a.T;
  unsigned n = 1;
  while (n < 8 && n < static_cast<unsigned>(a.B) && work > 4096LL * n) n *= 2;
  return launch_pdl(kv4_assign_kernel, dim3(n), kAssignThreads, smem, n, s, a);
}

cudaError_t launch_kv4_gather(const Kv4GatherArgs& a, cudaStream_t s) {
  const long long items = static_cast<long long>(a.B) * a.Hkv * (a.rows / kKv4Group + 2);
  const long long ctas = (items + 7) / 8;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ctas));
  switch (a.hd) {
    case 64: return launch_pdl(kv4_gather_kernel<64>, grid, 256, 0, 1, s, a);
    case 128: return launch_pdl(kv4_gather_kernel<128>, grid, 256, 0, 1, s, a);
    case 256: return launch_pdl(kv4_gather_kernel<256>, grid, 256, 0, 1, s, a);
    case 512: return launch_pdl(kv4_gather_kernel<512>, grid, 256, 0, 1, s, a);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace g4
