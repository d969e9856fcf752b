// Step a5 in bf16 with modified scores (g4_attn_prefill_mods): the MODS
// instantiations of the tcgen05 prefill.  What differs from g4_prefill_tc.cuh's
// account of the causal kernel:
//   * Every row has its own interval of keys.  The producer, which draws the
//     work items ahead of their use, reads the 128 rows' intervals and hands the
//     keys that some row sees on with the item, so tiles that no row sees are
//     neither loaded nor computed (a row packed of documents costs the documents'
//     areas); each softmax thread holds its row's interval in registers.
//   * 16 softmax warps, a thread a quarter of a row (the causal kernel: 8 and halves), and a warp of its own that
//     sends outputs out.  With what follows, uncapped 2 x 4096 tokens of head_dim 64 / 128 / 256 take 63 / 72 / 97 us
//     (the causal kernel 71 / 73 / 98).
//   * A thread reads its own part of a row only, since capping or biasing the rest too, for its maximum, would cost
//     more than to exchange maxima where the base has to be raised.
//   * The next item's intervals are read while the current one's output is finished, so that items of few tiles, as
//     of documents, do not wait for them.
//   * Rows of V outside of the item's keys are zeroed before they meet P, and rows of the output that a NaN or an
//     infinity reached from keys that other rows of the tile see are formed again (row_again; the check costs 1-2 %).
// Measured: a row of 8192 packed tokens (sliding, head_dim 256) 51 us, 61 with 8 warps and their exchange per tile;
// 4 x 2048 tokens with images, capped (head_dim 512) 174 us against 188; 2 x 4096 with a bias (head_dim 128) 75 against 87.
//   Not taken: groups of softmax warps that take key tiles in turn, so that one computes while the other waits.  Two
// groups of 8, two threads a row: 94 us for 2 x 4096 biased tokens of head_dim 128 against 75; of 4, a thread a row: 104.
// A group then has half of the issue slots for its tile, and its next scores wait for its weights and two products.
//   What bounds it: at head_dim 512 and 256 the tensor pipe and the issue of its instructions (half of the time, per tile
// 3600 of 5000 cycles at 512), at 128 and below the softmax's chain of load, maximum, exponentials and store
// (some 1700 cycles a tile, 2700 capped, of which 512 are the special-function unit's; issue slots are 58 % busy).
#include "g4_prefill_tc.cuh"

namespace g4 {
namespace {

template <int HD>
cudaError_t launch_mods_hd(const ModsTcArgs& a, cudaStream_t s) {
  const bool cap = a.cap_log2 > 0.0f, bias = a.slopes != nullptr;
  if (cap && bias) return launch_hd<HD, kMods, true, true>(a, s);
  if (cap) return launch_hd<HD, kMods, true, false>(a, s);
  if (bias) return launch_hd<HD, kMods, false, true>(a, s);
  return launch_hd<HD, kMods, false, false>(a, s);
}

}  // namespace

cudaError_t launch_prefill_mods(const ModsTcArgs& a_in, cudaStream_t s) {
  ModsTcArgs a = a_in;
  const cudaError_t e = take_prefill_counters(&a.item_ctr);
  if (e != cudaSuccess) return e;
  switch (a.hd) {
    case 64: return launch_mods_hd<64>(a, s);
    case 128: return launch_mods_hd<128>(a, s);
    case 256: return launch_mods_hd<256>(a, s);
    case 512: return launch_mods_hd<512>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace g4
