// Step a5 in bf16 with modified scores (g4_attn_prefill_mods): the MODS
// instantiations of the tcgen05 prefill.  What differs from g4_prefill_tc.cuh's
// account of the causal kernel:
//   * Every row has its own interval of keys.  The producer, which draws the
//     work items ahead of their use, reads the 128 rows' intervals and hands the
//     keys that some row sees on with the item, so tiles that no row sees are
//     neither loaded nor computed (a row packed of documents costs the documents'
//     areas); each softmax thread holds its row's interval in registers.
//   * A thread reads its half of a row only, since capping or biasing the other
//     half too, for its maximum, would cost more than an exchange: the halves'
//     maxima meet in shared memory, at the barrier that already tells that both
//     warps have read the tile.
//   * Rows of V outside of the item's keys are zeroed before they meet P.
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
