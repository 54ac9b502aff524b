"""The kernels that may start before the stream's previous kernel has ended, behind a kernel that lets its
dependents start at once and then takes longer than the bounded waits allow (2.5 s against 2 s), with the tokens,
weights and pool rows written at its end: nothing is read early, and no wait runs out meanwhile.  (The previous
kernel is compiled here; it ends by the clock and by an iteration count.)"""
import ctypes
import subprocess

import pytest
import torch

import gated_deltanet_mixer_gdn_b200 as gdn
from gated_deltanet_mixer_gdn_b200 import build
from gated_deltanet_mixer_gdn_b200.synth import Dims

pytestmark = pytest.mark.gpu
DIMS = Dims(num_k_heads=2, num_v_heads=4)

SLOW = r"""
#include <cuda_runtime.h>
#include <stdint.h>
__global__ void slow(uint4* dst, const uint4* src, size_t n, uint64_t ns) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (int i = 0; i < 5000000; ++i) {  // at least 1 us each
        __nanosleep(1000);
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t - t0 > ns) break;
    }
    for (size_t i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src[i];
}
extern "C" int run_slow(void* dst, const void* src, size_t bytes, uint64_t ns, void* stream) {
    slow<<<1, 256, 0, (cudaStream_t)stream>>>((uint4*)dst, (const uint4*)src, bytes / 16, ns);
    return (int)cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def slow_copy(tmp_path_factory):
    """copy(dst, src): src into dst, 2.5 s later, on the current stream."""
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    where = tmp_path_factory.mktemp("slow")
    (where / "slow.cu").write_text(SLOW)
    lib = str(where / "slow.so")
    subprocess.run([build.nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-O2", "-Xcompiler", "-fPIC", "-shared",
                    str(where / "slow.cu"), "-o", lib], check=True, timeout=300)
    fn = ctypes.CDLL(lib).run_slow
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint64, ctypes.c_void_p]

    def copy(dst, src):
        n = dst.numel() * dst.element_size()
        assert n % 16 == 0 and n == src.numel() * src.element_size()
        assert fn(dst.data_ptr(), src.data_ptr(), n, 2_500_000_000, torch.cuda.current_stream().cuda_stream) == 0

    return copy


@pytest.mark.parametrize("T", [1, 40, 100, 300])  # on chip, few tokens, more of them, pairs
def test_projection_behind_a_slow_kernel(slow_copy, T):
    dev = torch.device("cuda", 0)
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, DIMS.value_width), generator=g).to(torch.bfloat16).to(dev)
    w = gdn.quantize(torch.randn((320, DIMS.value_width), generator=g).to(torch.bfloat16).to(dev))
    want = gdn.out_proj_quant(x, w, dims=DIMS)
    late, out = torch.zeros_like(x), torch.zeros_like(want)
    torch.cuda.synchronize(dev)
    slow_copy(late, x)
    gdn.out_proj_quant(late, w, dims=DIMS, out=out)
    torch.cuda.synchronize(dev)
    assert gdn.last_device_error() == 0
    assert torch.equal(out, want)


def test_weights_behind_a_slow_kernel(slow_copy):
    """The codes arrive late; one token, so that the projection is the next kernel."""
    dev = torch.device("cuda", 0)
    g = torch.Generator().manual_seed(7)
    x = torch.randn((1, DIMS.value_width), generator=g).to(torch.bfloat16).to(dev)
    w = gdn.quantize(torch.randn((320, DIMS.value_width), generator=g).to(torch.bfloat16).to(dev))
    want = gdn.out_proj_quant(x, w, dims=DIMS)
    codes = torch.zeros_like(w.codes)
    late = gdn.QuantTensor(codes, w.scales, w.row_scale, w.format)
    torch.cuda.synchronize(dev)
    slow_copy(codes, w.codes)
    out = gdn.out_proj_quant(x, late, dims=DIMS)
    torch.cuda.synchronize(dev)
    assert gdn.last_device_error() == 0
    assert torch.equal(out, want)


def test_quantize_and_pool_behind_a_slow_kernel(slow_copy):
    dev = torch.device("cuda", 0)
    g = torch.Generator().manual_seed(8)
    x = torch.randn((40, 512), generator=g).to(torch.bfloat16).to(dev)
    want = gdn.dequantize(gdn.quantize(x))
    late = torch.zeros_like(x)
    torch.cuda.synchronize(dev)
    slow_copy(late, x)
    got = gdn.dequantize(gdn.quantize(late))
    state = torch.randn((3, DIMS.num_v_heads, 128, 128), generator=g).to(dev)
    conv = torch.randn((3, 3, DIMS.conv_channels), generator=g).to(dev)
    row = torch.randn(state[0].shape, generator=g).to(dev)
    before = state[1].clone()
    slow_copy(state[0], row)
    gdn.copy_slots([0, 1], [1, 2], state, conv, dims=DIMS)
    torch.cuda.synchronize(dev)
    assert gdn.last_device_error() == 0
    assert torch.equal(got, want)
    assert torch.equal(state[0], row) and torch.equal(state[1], row) and torch.equal(state[2], before)
