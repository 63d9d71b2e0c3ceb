"""Tensors whose element offsets pass 2^32: rows far apart in one large buffer give the same
results as the same rows next to one another."""
import pytest

import bit_weight_only_w4_b200 as w4
from tests import test_gpu_epilogue as epi
from tests.gpu_util import skip_without_gpu, torch_mod

pytestmark = pytest.mark.gpu

FAR = (1 << 32) + (1 << 24)   # elements of the buffer (8.6 GB of 16-bit ones)


def spread(buf, rows, width):
    """[rows, width] view of the buffer whose last row lies behind 2^32 elements."""
    step = (FAR - width) // (rows - 1) // 8 * 8
    assert step * (rows - 1) > 1 << 32
    return buf.as_strided((rows, width), (step, 1))


@pytest.fixture
def buf():
    skip_without_gpu()
    torch = torch_mod()
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB of free device memory")
    b = torch.empty(FAR, dtype=torch.float16, device="cuda")
    yield b
    del b
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M", [40, 130])
def test_product(buf, M):
    torch = torch_mod()
    L = epi.Layer(1, 256, 512, 128)
    X = L.acts(M)
    far = spread(buf, M, 256)
    near = torch.randn(M, 256, device="cuda").half()
    far.copy_(near)
    want = w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, 128, activation="silu", residual=near)
    w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, 128, activation="silu", residual=far, Y=far)
    assert torch.equal(far, want)


@pytest.mark.parametrize("dim", [64, 30])
def test_rope(buf, dim):
    torch = torch_mod()
    T, H = 50, 3
    near = torch.randn(T, H, dim, device="cuda").half()
    far = spread(buf, T, H * dim).unflatten(1, (H, dim))
    far.copy_(near)
    pos = torch.arange(T, device="cuda").int()
    inv = torch.rand(dim // 2, dtype=torch.float64, device="cuda")
    w4.w4_rope(far, pos, inv, Y=far)
    assert torch.equal(far, w4.w4_rope(near, pos, inv))


@pytest.mark.parametrize("tokens,keys", [(300, 300), (2, 700)])
def test_attention(buf, tokens, keys):
    torch = torch_mod()
    H, HK, D = 4, 2, 64
    q = torch.randn(tokens, H, D, device="cuda").half()
    k, v = (torch.randn(keys, HK, D, device="cuda").half() for _ in range(2))
    want = w4.w4_prompt_attention(q, k, v)
    kv = spread(buf, keys, 2 * HK * D).unflatten(1, (2 * HK, D))
    kv[:, :HK].copy_(k)
    kv[:, HK:].copy_(v)
    assert torch.equal(w4.w4_prompt_attention(q, kv[:, :HK], kv[:, HK:]), want)
    out = spread(buf, tokens, H * D).unflatten(1, (H, D))   # (the keys are not needed any more)
    w4.w4_prompt_attention(q, k, v, O=out)
    assert torch.equal(out, want)
    w4.w4_check_device_error()
