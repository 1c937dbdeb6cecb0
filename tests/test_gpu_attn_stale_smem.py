"""The readouts' results do not depend on what earlier kernels left in shared
memory, also when their code and data are cold in the caches."""
import ctypes
import subprocess

import pytest
import torch

from test_gpu_cache_dense import D, H, c2, entries, gen, prefix_inputs, queries, run_cross, run_prefix  # noqa: F401

pytestmark = pytest.mark.gpu

BYTES = 232448   # shared memory of one CTA: one CTA per SM at a time
SOURCE = """
#include <cuda_runtime.h>
#include <cstdint>
__global__ void fill(uint32_t v, uint32_t *sink) {
  extern __shared__ uint32_t s[];
  for (int i = threadIdx.x; i < %d / 4; i += blockDim.x) s[i] = v;
  __syncthreads();
  if (s[(threadIdx.x * 977) %% (%d / 4)] != v) *sink = 1;
}
extern "C" int fill_shared(uint32_t v, uint32_t *sink, int blocks, void *stream) {
  cudaFuncSetAttribute(fill, cudaFuncAttributeMaxDynamicSharedMemorySize, %d);
  fill<<<blocks, 1024, %d, (cudaStream_t)stream>>>(v, sink);
  return cudaGetLastError();
}
""" % (BYTES, BYTES, BYTES, BYTES)


@pytest.fixture(scope="module")
def stale(c2, tmp_path_factory):  # noqa: F811
    """A function that leaves a value in every SM's shared memory, with the
    caches full of other code and data."""
    from sparse_attention_fp4_csa2_gb300.build import ARCH, _nvcc
    d = tmp_path_factory.mktemp("fill")
    (d / "fill.cu").write_text(SOURCE)
    subprocess.run([_nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", str(d / "fill.cu"), "-o", str(d / "fill.so")], check=True)
    lib = ctypes.CDLL(str(d / "fill.so"))
    sink = torch.zeros(1, dtype=torch.int32, device="cuda")
    big = torch.zeros(1 << 27, device="cuda")
    mat = torch.randn(512, 512, device="cuda")
    blocks = 4 * torch.cuda.get_device_properties(0).multi_processor_count

    def run(value):
        for f in (torch.sin, torch.erfinv, torch.lgamma, torch.special.i0e, lambda x: x @ x, lambda x: torch.softmax(x, -1),
                  lambda x: torch.cumsum(x, 0), lambda x: x.double() @ x.double(), lambda x: torch.sort(x).values):
            f(mat)
        big.add_(1.0)
        assert lib.fill_shared(ctypes.c_uint32(value), ctypes.c_void_p(sink.data_ptr()), blocks,
                               ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    return run


# zeros, NaNs (as fp32 and as fp16), the largest finite values, all ones
VALUES = (0, 0x7FC07E00, 0x7F7F7BFF, 0xFFFFFFFF)


def same_each_time(stale, call, times=24):
    first = call()
    for i in range(times):
        stale(VALUES[i % len(VALUES)])
        for got, want in zip(call(), first):
            assert torch.equal(got, want), f"differs after shared memory held {VALUES[i % len(VALUES)]:#x}"
    assert all(torch.isfinite(x).any() for x in first)


@pytest.mark.parametrize("own", [
    [(0, 0), (512, 1), (1, 128), (512, 128)],   # chunks without keys, and a sequence without any
    [(300, 77)], [(0, 128)] * 2, [(512, 128)] * 16])
@pytest.mark.parametrize("kernel", [1, 2])
def test_sparse_attn(c2, stale, own, kernel):  # noqa: F811
    p, q, _, kv, idx, swa, sc, sl = prefix_inputs(c2, len(own), 0, 512, 128, 7, own)
    p = c2.Params.make(attn_kernel=kernel)
    ws = c2.workspace(c2.OP_ATTN, len(own), kv.shape[1], p)

    def call():
        out = torch.full((len(own), H, D), 3.0, device="cuda")
        lse = torch.full((len(own), H), 3.0, device="cuda")
        c2.sparse_attn(p, q, kv, idx, swa, sc, sl, out, ws, lse=lse)
        return out, lse
    same_each_time(stale, call)
    out, lse = call()
    for b, (k, w) in enumerate(own):
        assert torch.isfinite(out[b]).all()
        if k + w == 0:
            assert (out[b] == 0).all() and torch.isneginf(lse[b]).all()


def test_prefix_attn(c2, stale):  # noqa: F811
    args = prefix_inputs(c2, 4, 700, 512, 128, 8, [(0, 0), (512, 1), (1, 128), (512, 128)])
    same_each_time(stale, lambda: run_prefix(c2, *args))


@pytest.mark.parametrize("n_q,lens", [(1, [1000, 0, 1, 257]), (3, [256, 30, 513, 2000]), (40, [700, 0, 255, 300])])
def test_cross_attn(c2, stale, n_q, lens):  # noqa: F811
    kv = entries(c2, 4 * 2000, 9).view(4, 2000, -1)
    q = queries((4, n_q), 10)
    nv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    same_each_time(stale, lambda: run_cross(c2, q, kv, nv, max(lens)))
