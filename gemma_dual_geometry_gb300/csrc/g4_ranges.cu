// The interval of keys that each token sees (g4_attn_visible_ranges), from runs
// of equal ids: a document's first position D, a span's first and last + 1, S and E.
//
// A position p is a cut of the documents where doc[p] != doc[p - 1] (or p = 0),
// and a cut of the spans where it is one of the documents or span[p] !=
// span[p - 1].  D and S are the last cuts at or before p (running maxima of the
// cuts' positions), E the first cut of the spans after p (a running minimum from
// the other end), or seq_lens[b].
//
// One cluster per sequence.  Its CTAs share out the positions in tiles of
// kTile; each first finds the last and first cuts of its tiles, hands them to
// the others through distributed shared memory, and then scans its tiles with
// what came before and comes after.  A CTA of one tile keeps the ids in registers
// between the two passes.
//   Bound by latency: load, reduction, cluster barrier, scan, store: 8 rows of 32768
// positions (3.7 MB) 5.9 us, one of 1000 3.0 us, one of 131072 12 us.  (CTAs that find what
// they need of the rest of the row by themselves, looking back for the beginning of their
// run, took 18, 3.7 and 68 us.)
#include <cooperative_groups.h>

#include "g4_device.cuh"
#include "g4_internal.h"

namespace g4 {
namespace {

namespace cg = cooperative_groups;

// (1024 threads of 4 positions: 6.4 us against 5.9 at 8 rows of 32768; 256 of 16: 6.2)
constexpr int kRangesThreads = 512;
constexpr int kRangesMaxTiles = 512;             // tiles per CTA: 2^24 positions over 8 CTAs, where no cluster of 16 is to be had
constexpr int kNone = 0x7fffffff;

// One tile's ids of this thread (kPer consecutive positions), and what is a cut.
template <int kPer>
struct Ids {
  int doc[kPer], span[kPer];
  uint32_t doc_cut, span_cut;  // bit i: position i of the thread's is a cut
};

// Three numbers of a tile: its last cuts (-1: none) and its first cut of the spans (kNone).
struct Cuts {
  int doc, span, first;
};

__device__ __forceinline__ Cuts no_cuts() { return {-1, -1, kNone}; }
__device__ __forceinline__ Cuts join(Cuts a, Cuts b) {
  return {max(a.doc, b.doc), max(a.span, b.span), min(a.first, b.first)};
}

template <int kPer>
__global__ void __launch_bounds__(kRangesThreads) ranges_kernel(const __grid_constant__ RangesArgs a) {
  __shared__ Cuts s_tile[kRangesMaxTiles];  // of this CTA's tiles
  __shared__ Cuts s_cta;                    // of all of them
  constexpr int NW = kRangesThreads / 32;
  constexpr int kTile = kRangesThreads * kPer;
  static_assert(kPer == 4 || 8LL * kTile * kRangesMaxTiles >= 1 << 24, "longest rows");
  __shared__ Cuts s_warp[NW];
  __shared__ int2 s_out[kTile + kTile / 32];  // intervals of a tile
  cg::cluster_group cluster = cg::this_cluster();
  const int nctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int b = blockIdx.x / nctas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr unsigned kAll = 0xffffffffu;

  pdl_wait();
  pdl_trigger();
  const int len = min(max(a.lens[b], 0), a.max_len);
  const int start = min(max(a.q_start[b], -a.T), 0x7fffffff - a.T);
  const int* doc = a.doc != nullptr ? a.doc + static_cast<size_t>(b) * a.max_len : nullptr;
  const int* span = a.span != nullptr ? a.span + static_cast<size_t>(b) * a.max_len : nullptr;
  const int ntiles = (len + kTile - 1) / kTile;
  const int per_cta = (ntiles + nctas - 1) / nctas;
  const int t0 = min(ntiles, rank * per_cta), t1 = min(ntiles, t0 + per_cta);

  // Ids of the thread's positions of a tile; those from len on take no part.
  auto load = [&](int tile) {
    Ids<kPer> d;
    const int p0 = tile * kTile + tid * kPer;
    d.doc_cut = d.span_cut = 0;
    int before_doc = 0, before_span = -1;
    if (p0 > 0 && p0 < len) {
      if (doc != nullptr) before_doc = __ldg(doc + p0 - 1);
      if (span != nullptr) before_span = __ldg(span + p0 - 1);
    }
    if (a.aligned_ids && p0 + kPer <= len) {
#pragma unroll
      for (int i = 0; i < kPer; i += 4) {
        const int4 x = doc != nullptr ? __ldg(reinterpret_cast<const int4*>(doc + p0 + i)) : make_int4(0, 0, 0, 0);
        const int4 y = span != nullptr ? __ldg(reinterpret_cast<const int4*>(span + p0 + i)) : make_int4(-1, -1, -1, -1);
        d.doc[i] = x.x; d.doc[i + 1] = x.y; d.doc[i + 2] = x.z; d.doc[i + 3] = x.w;
        d.span[i] = y.x; d.span[i + 1] = y.y; d.span[i + 2] = y.z; d.span[i + 3] = y.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int p = p0 + i;
        d.doc[i] = doc != nullptr && p < len ? __ldg(doc + p) : 0;
        d.span[i] = span != nullptr && p < len ? __ldg(span + p) : -1;
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = p0 + i;
      if (p >= len) continue;
      const bool dc = p == 0 || d.doc[i] != (i == 0 ? before_doc : d.doc[i - 1]);
      const bool sc = dc || d.span[i] != (i == 0 ? before_span : d.span[i - 1]);
      d.doc_cut |= static_cast<uint32_t>(dc) << i;
      d.span_cut |= static_cast<uint32_t>(sc) << i;
    }
    return d;
  };
  auto of_thread = [&](const Ids<kPer>& d, int tile) {
    const int p0 = tile * kTile + tid * kPer;
    Cuts c = no_cuts();
    if (d.doc_cut) c.doc = p0 + 31 - __clz(d.doc_cut);
    if (d.span_cut) {
      c.span = p0 + 31 - __clz(d.span_cut);
      c.first = p0 + __ffs(d.span_cut) - 1;
    }
    return c;
  };
  auto of_warp = [&](Cuts c) {
    return Cuts{__reduce_max_sync(kAll, c.doc), __reduce_max_sync(kAll, c.span), __reduce_min_sync(kAll, c.first)};
  };

  // First pass: the cuts of each tile of this CTA.
  Ids<kPer> ids = {};
  for (int tile = t0; tile < t1; ++tile) {
    ids = load(tile);
    const Cuts c = of_warp(of_thread(ids, tile));
    if (lane == 0) s_warp[warp] = c;
    __syncthreads();
    if (warp == 0) {
      const Cuts all = of_warp(lane < NW ? s_warp[lane] : no_cuts());
      if (lane == 0) s_tile[tile - t0] = all;
    }
    __syncthreads();
  }
  if (warp == 0) {
    Cuts c = no_cuts();
    for (int i = lane; i < t1 - t0; i += 32) c = join(c, s_tile[i]);
    c = of_warp(c);
    if (lane == 0) s_cta = c;
  }
  Cuts before = no_cuts(), after = no_cuts();  // of the CTAs before and after this one
  if (nctas > 1) {
    cluster.sync();
    for (int r = 0; r < nctas; ++r) {
      const Cuts* other = cluster.map_shared_rank(&s_cta, r);
      if (r < rank) before = join(before, *other);
      if (r > rank) after = join(after, *other);
    }
    cluster.barrier_arrive();  // (nobody leaves while others read its cuts)
  }

  // Second pass: the tiles' tokens.
  for (int tile = t0; tile < t1; ++tile) {
    const int tile_begin = tile * kTile, tile_end = min(len, tile_begin + kTile);
    const bool wanted = tile_begin < static_cast<long long>(start) + a.T && tile_end > start;  // (the same for all threads)
    if (wanted) {
      if (t1 - t0 > 1) ids = load(tile);
      Cuts far = after;  // first cut behind this tile
      for (int i = tile + 1; i < t1; ++i) far = join(far, s_tile[i - t0]);
      // scans: last cuts of the threads before, first cut of the threads behind
      const Cuts own = of_thread(ids, tile);
      Cuts scan = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int d = __shfl_up_sync(kAll, scan.doc, o), s = __shfl_up_sync(kAll, scan.span, o);
        const int f = __shfl_down_sync(kAll, scan.first, o);
        if (lane >= o) {
          scan.doc = max(scan.doc, d);
          scan.span = max(scan.span, s);
        }
        if (lane + o < 32) scan.first = min(scan.first, f);
      }
      __syncthreads();  // (s_warp is free again)
      if (lane == 31) {
        s_warp[warp].doc = scan.doc;
        s_warp[warp].span = scan.span;
      }
      if (lane == 0) s_warp[warp].first = scan.first;
      __syncthreads();
      const Cuts others = lane < NW ? s_warp[lane] : no_cuts();
      const Cuts w_before = of_warp(lane < warp ? others : no_cuts());
      const Cuts w_after = of_warp(lane > warp ? others : no_cuts());
      int d = __shfl_up_sync(kAll, scan.doc, 1), s = __shfl_up_sync(kAll, scan.span, 1);
      int e = __shfl_down_sync(kAll, scan.first, 1);
      if (lane == 0) d = s = -1;
      if (lane == 31) e = kNone;
      d = max(max(d, w_before.doc), before.doc);
      s = max(max(s, w_before.span), before.span);
      e = min(min(e, w_after.first), far.first);
      e = min(e, len);
      int ends[kPer];
#pragma unroll
      for (int i = kPer - 1; i >= 0; --i) {
        ends[i] = e;
        if (ids.span_cut >> i & 1) e = tile_begin + tid * kPer + i;
      }
      int first[kPer], last[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int p = tile_begin + tid * kPer + i;
        if (ids.doc_cut >> i & 1) d = p;
        if (ids.span_cut >> i & 1) s = p;
        first[i] = a.window > 0 ? max(d, p - a.window + 1) : d;
        last[i] = p + 1;
        if (ids.span[i] >= 0) {
          first[i] = min(first[i], s);
          last[i] = ends[i];
        }
        if (ids.doc[i] < 0) first[i] = last[i] = 0;
      }
      const int p0 = tile_begin + tid * kPer;
      const long long t = static_cast<long long>(p0) - start;  // the first one's token
      int* const to_begin = a.begin + static_cast<size_t>(b) * a.T + t;
      int* const to_end = a.end + static_cast<size_t>(b) * a.T + t;
      if (a.aligned_out && (start & 3) == 0) {
        if (t >= 0 && t + kPer <= a.T && p0 + kPer <= len) {
#pragma unroll
          for (int i = 0; i < kPer; i += 4) {
            *reinterpret_cast<int4*>(to_begin + i) = make_int4(first[i], first[i + 1], first[i + 2], first[i + 3]);
            *reinterpret_cast<int4*>(to_end + i) = make_int4(last[i], last[i + 1], last[i + 2], last[i + 3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            if (p0 + i < len && t + i >= 0 && t + i < a.T) {
              to_begin[i] = first[i];
              to_end[i] = last[i];
            }
          }
        }
      } else {
        // rows that are not written four at a time: neighbours by neighbouring threads (44 x 5691 tokens 6.4 us, 9.5 by
        // each thread its own)
        auto slot = [](int i) { return i + i / 32; };
        __syncthreads();  // (the tile before has been written)
#pragma unroll
        for (int i = 0; i < kPer; ++i) s_out[slot(tid * kPer + i)] = make_int2(first[i], last[i]);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int at = i * kRangesThreads + tid;
          const long long u = static_cast<long long>(tile_begin + at) - start;
          if (tile_begin + at < len && u >= 0 && u < a.T) {
            const int2 v = s_out[slot(at)];
            a.begin[static_cast<size_t>(b) * a.T + u] = v.x;
            a.end[static_cast<size_t>(b) * a.T + u] = v.y;
          }
        }
      }
    }
    before = join(before, s_tile[tile - t0]);
  }
  // tokens that are no position held
  for (long long t = rank * kRangesThreads + tid; t < a.T; t += nctas * kRangesThreads) {
    const int p = start + static_cast<int>(t);
    if (p < 0 || p >= len) {
      const size_t at = static_cast<size_t>(b) * a.T + t;
      a.begin[at] = 0;
      a.end[at] = 0;
    }
  }
  if (nctas > 1) cluster.barrier_wait();
}

template <int kPer>
cudaError_t launch_per(const RangesArgs& a, unsigned nctas, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * nctas);
  cfg.blockDim = dim3(kRangesThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = nctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, ranges_kernel<kPer>, a);
}

}  // namespace

cudaError_t launch_ranges(const RangesArgs& a_in, cudaStream_t s) {
  RangesArgs a = a_in;
  auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  a.aligned_ids = a.max_len % 4 == 0 && aligned(a.doc) && aligned(a.span);
  a.aligned_out = a.T % 4 == 0 && aligned(a.begin) && aligned(a.end);
  // A CTA per tile of the longest row, up to a cluster of 16 where that may be had.  Rows of one tile of 2048 take that one
  // (1000 positions 3.0 us against 3.6 with a tile of 4096).
  if (a.max_len <= 4 * kRangesThreads) return launch_per<4>(a, 1, s);
  unsigned nctas = 1;
  const unsigned most = a.max_len > 8 * 8 * kRangesThreads ? cluster_limit_once<ranges_kernel<8>>(kRangesThreads, 0) : 8;
  while (nctas < most && static_cast<long long>(nctas) * 8 * kRangesThreads < a.max_len) nctas *= 2;
  return launch_per<8>(a, nctas, s);
}

}  // namespace g4
