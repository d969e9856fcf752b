// Steps a6 and a5 in float32 on CUDA cores: the instantiations of
// g4_attn_simt.cuh, and the decode's split plan.
#include "g4_attn_simt.cuh"

namespace g4 {

cudaError_t launch_attn_simt(const AttnSimtArgs& a, int dtype, cudaStream_t s) {
  return dtype == 1 ? launch_simt_t<__nv_bfloat16, false>(a, s) : launch_simt_t<float, false>(a, s);
}

int sm_count() {
  static int cached[128] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) {
    cudaGetLastError();
    return 152;  // GB300
  }
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = 152;
    }
    cached[dev] = n;
  }
  return cached[dev];
}

DecodePlan decode_plan(int dtype, int sliding, int window, int hd, int H, int Hkv, int B, int max_seq_len) {
  DecodePlan p;
  const int span = sliding ? (max_seq_len < window ? max_seq_len : window) : max_seq_len;
  if (decode_win_eligible(dtype, hd, H / Hkv, span, B * Hkv)) {
    p.win = 1;
    p.chunk = 64;
    p.nsplit = decode_win_splits(span);
    p.o_bytes = p.m_bytes = p.t_bytes = p.ws_bytes = 0;
    return p;
  }
  p.win = 0;
  const int units = B * Hkv;
  const int G = H / Hkv;
  // CTA slots of one wave: SMs x CTAs per SM (two for G*hd >= 2048, else three).
  const int slots = sm_count() * ((G * hd >= 2048) ? 2 : 3);
  // Splits: at least 64 keys each, and at most sqrt(span / 8) so that the
  // final merge (nsplit partials of G*hd floats) stays small next to the keys
  // each split streams; within that, a whole number of waves (4 down to 1).
  const int by_len = (span + 63) / 64;
  int by_merge = static_cast<int>(sqrt(static_cast<double>(span) / 8.0));
  if (by_merge < 4) by_merge = 4;
  int cap = by_len < by_merge ? by_len : by_merge;
  if (cap > kMaxSplits) cap = kMaxSplits;
  if (cap < 1) cap = 1;
  int nsplit = 0;
  if (units * 2 <= sm_count()) {
    // Few (row, kv head) units: one 8-warp CTA per SM, as many splits as fit
    // one wave, so each CTA streams a long key range and the per-CTA work
    // (norm, merges) is paid as few times as possible.
    nsplit = sm_count() / units;
    if (nsplit > cap) nsplit = cap;
  }
  for (int m = 4; m >= 1 && nsplit == 0; --m) {
    const int ns = static_cast<int>((static_cast<long long>(m) * slots) / units);
    if (ns >= 1 && ns <= cap) nsplit = ns;
  }
  if (nsplit == 0) {
    const int want = (slots + units - 1) / units;
    nsplit = want < cap ? want : cap;
  }
  if (nsplit < 1) nsplit = 1;
  int chunk = (span + nsplit - 1) / nsplit;
  chunk = (chunk + 15) / 16 * 16;
  nsplit = (span + chunk - 1) / chunk;
  p.chunk = chunk;
  p.nsplit = nsplit;
  if (nsplit <= 1) {
    p.o_bytes = p.m_bytes = p.t_bytes = p.ws_bytes = 0;
  } else {
    const size_t np = static_cast<size_t>(B) * H * nsplit;
    p.o_bytes = (np * hd * 4 + 255) / 256 * 256;
    p.m_bytes = (np * 4 + 255) / 256 * 256;
    p.t_bytes = (static_cast<size_t>(B) * Hkv * 4 + 255) / 256 * 256;
    p.ws_bytes = p.o_bytes + 2 * p.m_bytes + p.t_bytes;
  }
  return p;
}

}  // namespace g4
