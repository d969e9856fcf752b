// Prefill in float32 with modified scores (g4_attn_prefill_mods): the MODS instantiations of the split-KV kernel.
#include "g4_attn_simt.cuh"

namespace g4 {

cudaError_t launch_attn_simt_mods(const ModsSimtArgs& a, cudaStream_t s) { return launch_simt_t<float, true>(a, s); }

}  // namespace g4
