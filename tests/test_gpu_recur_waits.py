"""The recurrence's hand-off waits where one of them runs out: a small kernel around the exchange of
gla_recur.cuh, one of whose warps stops giving maps.  Every wait in it ends by its limit."""
import ctypes
import os
import subprocess

import pytest
import torch

from gated_linear_attention_gla_gb300 import build as glabuild

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "gla_recur.cuh"
using namespace gla;
using namespace gla::recur;
// One computing warp and the exchange warp in each of one or four blocks; h -> h / 2 + 1 a step and block.
__global__ void alone(RecurArgs a, int steps, int bad_step, float* out) {
  __shared__ Maps maps;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  maps_init(maps, 1, 1);
  if (w == 1) {
    const f32x2 h = exchange_alone<false>(maps, steps, 1, lane, both(0.f), a);
    if (lane == 0) out[0] = h.x;
  } else {
    for (int step = 0; step < steps; ++step) {
      if (step == bad_step) break;
      give(maps, step, 0, lane, make_float4(0.5f, 0.5f, 1.f, 1.f));
      if (take(maps, step, 0, lane, a.status).x > 2.f) break;
    }
  }
}
__global__ void __cluster_dims__(4, 1, 1) walk(RecurArgs a, int steps, int bad_rank, int bad_step, float* out) {
  __shared__ Maps maps;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, rank = blockIdx.x & 3;
  maps_init(maps, 1, 4);
  Came came;
  if (w == 1) {
    const f32x2 h = exchange<false>(maps, steps, 1, rank, 4, lane, both(0.f), a, came);
    if (lane == 0) out[rank] = h.x;
  } else {
    for (int step = 0; step < steps; ++step) {
      if (rank == bad_rank && step == bad_step) break;
      give(maps, step, 0, lane, make_float4(0.5f, 0.5f, 1.f, 1.f));
      if (take(maps, step, 0, lane, a.status).x > 2.f) break;
    }
  }
  part(maps, w == 1, lane, rank, 4, came);
}
extern "C" int run(unsigned* status, unsigned long long limit, int steps, int bad_rank, int bad_step, float* out) {
  RecurArgs a{};
  a.status = status;
  a.wait_ns = limit;
  if (bad_rank == -2) alone<<<1, 64>>>(a, steps, bad_step, out);
  else walk<<<8, 64>>>(a, steps, bad_rank, bad_step, out);
  return (int)cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    d = tmp_path_factory.mktemp("waits")
    src, out = str(d / "waits.cu"), str(d / "waits.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([glabuild._nvcc(), "-shared", "-o", out, src, "-O2", "-std=c++17", *glabuild.ARCH, "-Xcompiler",
                    "-fPIC", "-I", glabuild.INCLUDE, "-I", glabuild.CSRC, "--expt-relaxed-constexpr"], check=True)
    lib = ctypes.CDLL(os.path.abspath(out))
    lib.run.argtypes = [ctypes.c_void_p, ctypes.c_uint64] + [ctypes.c_int] * 3 + [ctypes.c_void_p]
    return lib


def test_recur_waits_run_out(probe):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(4, device="cuda")

    def call(limit, steps, bad_rank, bad_step):
        status.zero_()
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.default_stream().synchronize()
        a.record(torch.cuda.default_stream())
        assert probe.run(status.data_ptr(), limit, steps, bad_rank, bad_step, out.data_ptr()) == 0
        b.record(torch.cuda.default_stream())
        torch.cuda.synchronize()
        return int(status), a.elapsed_time(b)

    def right(steps):
        assert call(2_000_000_000, steps, -1, -1)[0] == 0
        assert out.tolist() == [2 - 2 ** (1 - 4.0 * steps)] * 4 or steps > 5  # exact in fp32 up to there

    right(5)
    right(1000)
    for bad_rank in range(4):
        for steps, bad_step in ((1, 0), (2, 1), (9, 0), (9, 1), (9, 2), (9, 7), (9, 8)):
            code, ms = call(1_000_000, steps, bad_rank, bad_step)
            # the limit, and the tests before and between readings of the time
            assert code != 0 and ms < 1000, (bad_rank, steps, bad_step, code, ms)
            right(5)
    # a block alone, whose exchange looks every 64 steps whether a wait ran out: each takes 256 tests until then
    assert call(2_000_000_000, 7, -2, -1)[0] == 0 and out.tolist()[0] == 2 - 2 ** -6
    for steps, bad_step in ((1, 0), (2, 1), (5, 1), (3, 2)):
        code, ms = call(1_000_000, steps, -2, bad_step)
        assert code != 0 and ms < 1000, (steps, bad_step, code, ms)
    code, ms = call(1_000_000, 100000, -2, 70)
    assert code != 0 and ms < 5000, (code, ms)
