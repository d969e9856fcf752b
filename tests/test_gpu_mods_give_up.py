"""Decode with modified scores after a wait for keys that gave up: the workspace serves the next call all the same.

The kernel is compiled here from its source with a wait that gives up at once in the CTA that a test names (the waits for
copies in flight, which follow, stay as they are)."""

import ctypes
import os
import subprocess

import pytest

from gemma_dual_geometry_gb300 import build as g4build
from gpu_common import DEV, W, torch
from test_gpu_mods import i32, unit

pytestmark = pytest.mark.gpu

HEAD = r"""
#define warp_wait warp_wait_in_full
#include "g4_device.cuh"
#undef warp_wait

namespace g4 {
// err[1]: the CTA whose second warp gives up
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int* err, volatile int* abort = nullptr) {
  if (err != nullptr && static_cast<int>(blockIdx.x) == err[1] && threadIdx.x / 32 == 1) {
    if (threadIdx.x % 32 == 0) atomicExch(err, kErrWaitTimeout);
    __syncwarp();
    return false;
  }
  return warp_wait_in_full(bar, parity, err, abort);
}
}  // namespace g4
"""

TAIL = r"""
}  // namespace
}  // namespace g4

extern "C" int decode(const void* q, const void* ck, const void* cv, void* out, const int* lens, uint8_t* ws, int* err, int B,
                      int Hkv, int max_len, int nctas, void* stream) {
  g4::ModsDecodeArgs a = {};
  a.q = q;
  a.ck = ck;
  a.cv = cv;
  a.out = out;
  a.lens = lens;
  a.err = err;
  a.B = B;
  a.H = 4 * Hkv;
  a.Hkv = Hkv;
  a.hd = 128;
  a.max_len = a.len_cap = max_len;
  a.nctas = nctas;
  a.scale_log2 = 0.5f;
  a.tickets = reinterpret_cast<unsigned*>(ws);
  a.ws_ml = reinterpret_cast<float2*>(ws + g4::kTicketBytes);
  a.ws_o = reinterpret_cast<float*>(ws + g4::kTicketBytes + 2 * nctas * 4 * sizeof(float2));
  return g4::launch_w<__nv_bfloat16, 128, 4, 4>(a, static_cast<cudaStream_t>(stream));
}
"""


@pytest.fixture(scope="module")
def decode(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    text = open(os.path.join(g4build.CSRC, "g4_decode_mods.cu")).read()
    kernel = text[:text.index("template <typename T, int HD, int G>\ncudaError_t launch_g(")]
    tmp = tmp_path_factory.mktemp("give_up")
    src, so = tmp / "give_up.cu", tmp / "give_up.so"
    src.write_text(HEAD + kernel + TAIL)
    subprocess.run([g4build.nvcc_path()] + g4build._flags() + ["-shared", "-cudart", "static", str(src), "-o", str(so)],
                   check=True)
    fn = ctypes.CDLL(str(so)).decode
    fn.argtypes = [ctypes.c_void_p] * 7 + [ctypes.c_int] * 4 + [ctypes.c_void_p]
    return fn


# lengths, CTAs: parts of 118 keys cut at units (40 of one sequence, two levels of merges), and shares of several units
@pytest.mark.parametrize("lens,nctas", [([4000, 100], 70), ([4000, 100], 5), ([700, 800, 20, 0, 900], 7), ([9000], 300)])
@pytest.mark.parametrize("victim", [0, 1, 3, 4])
def test_the_workspace_is_left_ready(decode, lens, nctas, victim):
    B, Hkv, n = len(lens), 2, max(lens)
    k, v = (unit((B, Hkv, n, 128), i, W.BF16).to(DEV) for i in (1, 2))
    q, d_lens = unit((B, 4 * Hkv, 128), 3, W.BF16).to(DEV), i32(lens)
    size = 3 * 2 * 1024 * 4
    ws = torch.zeros(size + 2 * nctas * 4 * (8 + 512), dtype=torch.uint8, device=DEV)

    def run(victim):
        out = torch.full_like(q, float("nan"))
        err = i32([0, victim])
        status = decode(*(x.data_ptr() for x in (q, k, v, out, d_lens, ws, err)), B, Hkv, n, nctas,
                        torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert status == 0 and (ws[:size] == 0).all()
        return out, int(err[0])

    want, error = run(-1)
    assert error == 0 and torch.isfinite(want).all()
    out, error = run(victim)
    assert error == 1 and torch.isfinite(out).all() and not torch.equal(out, want)
    out, error = run(-1)
    assert error == 0 and torch.equal(out, want)
