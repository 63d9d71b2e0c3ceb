"""More of the products with an epilogue: activations at the ends of their range."""
import math

import pytest

import bit_weight_only_w4_b200 as w4
from tests.gpu_util import skip_without_gpu, torch_mod
from tests.test_gpu_epilogue import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("activation", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype,out_dtype", [("float16", "float16"), ("bfloat16", "bfloat16"), ("bfloat16", "float32")])
@pytest.mark.parametrize("M", [3, 20, 70])
def test_infinite_and_large_arguments(M, dtype, out_dtype, activation):
    """A bias of +infinity gives +infinity, of 10^30 itself (infinity in fp16), of -10^30 zero
    (none: itself), NaN NaN; other columns keep their bits."""
    skip_without_gpu()
    torch = torch_mod()
    L = Layer(21, 96, 256, 64, dtype=dtype)
    X = L.acts(M)
    out = getattr(torch, out_dtype)
    run = lambda b, **k: w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, 64, bias=b, activation=activation, out_dtype=out, **k)  # noqa: E731
    zero = torch.zeros(96, device="cuda")
    bias = zero.clone()
    at = {3: math.inf, 12: 1e30, 33: -1e30, 40: math.nan}
    for n, v in at.items():
        bias[n] = v
    want = run(zero)
    for n, v in at.items():
        want[:, n] = torch.tensor(v if v != v or v > 0 or activation == "none" else 0.0).to(out)
    got = run(bias)
    rest = torch.ones(96, dtype=torch.bool, device="cuda")
    rest[list(at)] = False
    assert torch.equal(got[:, rest], want[:, rest])
    same = (got == want) | (got.isnan() & want.isnan())
    assert same.all(), [(n, got[0, n].item(), want[0, n].item()) for n in at]
    # gated: gate +infinity times up
    bias = zero.clone()
    bias[2] = math.inf
    y, plain = run(bias, gated=True), run(zero, gated=True)
    up = w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, 64, out_dtype=torch.float32)[:, 10]
    assert torch.equal(y[:, 2], torch.where(up > 0, math.inf, -math.inf).to(out))
    keep = torch.arange(48, device="cuda") != 2
    assert torch.equal(y[:, keep], plain[:, keep])
    w4.w4_check_device_error()
