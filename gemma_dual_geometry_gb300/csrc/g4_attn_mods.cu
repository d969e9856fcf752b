// Decode, and prefill in float32, with modified scores (g4_attn_decode_mods,
// g4_attn_prefill_mods): the MODS instantiations of the split-KV kernel.
#include "g4_attn_simt.cuh"

namespace g4 {

cudaError_t launch_attn_simt_mods(const ModsSimtArgs& a, int dtype, cudaStream_t s) {
  return dtype == 1 ? launch_simt_t<__nv_bfloat16, true>(a, s) : launch_simt_t<float, true>(a, s);
}

}  // namespace g4
