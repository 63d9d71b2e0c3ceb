"""Calls on a stream other than the current one that allocate their outputs: memory that was freed
on the current stream, and that work queued there still reads, is not theirs to write."""
import pytest

import bit_weight_only_w4_b200 as w4
from tests.gpu_util import skip_without_gpu, torch_mod
from tests.test_gpu_epilogue import Layer

pytestmark = pytest.mark.gpu


def cases():
    torch = torch_mod()
    L = Layer(1, 1024, 512, 128)
    X = L.acts(256)
    q = torch.randn(256, 4, 256, device="cuda").half()[:, :, :128]
    heads = torch.randn(512, 8, 128, device="cuda").half()
    pos, inv = torch.arange(512, device="cuda").int(), torch.rand(64, dtype=torch.float64, device="cuda")
    W = torch.randn(256, 2048, device="cuda").half()
    return {
        "gemm": lambda **k: w4.w4a16_gemm(X, L.qw, L.sc, L.zr, 128, **k),
        "gemm_epi": lambda **k: w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, 128, activation="silu", **k),
        "rope": lambda **k: w4.w4_rope(heads, pos, inv, **k),
        "attention": lambda **k: w4.w4_prompt_attention(q, q, q, **k),
        "quantize": lambda **k: w4.w4_quantize_pack(W, **k)[0],
    }


@pytest.mark.parametrize("name", ["gemm", "gemm_epi", "rope", "attention", "quantize"])
def test_output_does_not_take_memory_in_use_on_the_current_stream(name):
    skip_without_gpu()
    torch = torch_mod()
    call = cases()[name]
    want = call()
    size = want.numel() * want.element_size()
    s = torch.cuda.Stream()
    call(stream=s)                       # (first use of the stream and of its workspace)
    torch.cuda.synchronize()
    copy = torch.zeros(size, dtype=torch.uint8, device="cuda")
    old = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)       # about a tenth of a second
    copy.copy_(old)
    del old                              # its block is the next one of that size
    got = call(stream=s)
    torch.cuda.synchronize()
    assert bool((copy == 7).all()) and torch.equal(got, want)


@pytest.mark.parametrize("name", ["gemm", "gemm_epi", "rope", "attention", "quantize"])
def test_output_is_kept_while_the_current_stream_reads_it(name):
    skip_without_gpu()
    torch = torch_mod()
    call = cases()[name]
    want = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    copy = torch.zeros_like(got)
    torch.cuda._sleep(200_000_000)
    copy.copy_(got)
    size = got.numel() * got.element_size()
    del got
    with torch.cuda.stream(s):
        torch.full((size,), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
