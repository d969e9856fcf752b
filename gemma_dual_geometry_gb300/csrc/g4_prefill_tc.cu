// Step a5 in bf16 on the tensor cores, causal and encoder form: the
// instantiations of g4_prefill_tc.cuh, and the counters of all its launches.
#include <mutex>

#include "g4_prefill_tc.cuh"

namespace g4 {

// Work-item counters of the persistent prefill, one pair per launch in flight
// (launches take the pairs in turn, so up to kCtrSlots launches may overlap).
constexpr int kCtrSlots = 64;
__device__ unsigned g_prefill_ctr[kCtrSlots][2];

cudaError_t take_prefill_counters(unsigned** ctr) {
  static std::mutex mu;
  static unsigned* base[128] = {};
  static unsigned next_slot = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (base[dev] == nullptr) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_prefill_ctr);
    if (e != cudaSuccess) return e;
    base[dev] = static_cast<unsigned*>(p);
  }
  *ctr = base[dev] + 2 * (next_slot++ % kCtrSlots);
  return cudaSuccess;
}

cudaError_t launch_prefill_tc(const PrefillTcArgs& a_in, cudaStream_t s) {
  PrefillTcArgs a = a_in;
  const cudaError_t e = take_prefill_counters(&a.item_ctr);
  if (e != cudaSuccess) return e;
  if (a.bidir) {
    switch (a.hd) {
      case 64: return launch_hd<64, kBidir>(a, s);
      case 128: return launch_hd<128, kBidir>(a, s);
      case 256: return launch_hd<256, kBidir>(a, s);
      case 512: return launch_hd<512, kBidir>(a, s);
      default: return cudaErrorInvalidValue;
    }
  }
  switch (a.hd) {
    case 64: return launch_hd<64, kCausal>(a, s);
    case 128: return launch_hd<128, kCausal>(a, s);
    case 256: return launch_hd<256, kCausal>(a, s);
    case 512: return launch_hd<512, kCausal>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace g4
