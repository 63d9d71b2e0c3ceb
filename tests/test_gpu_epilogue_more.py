"""More of the products with an epilogue: activations at the ends of their range, and the calls
that run as two products, in every form a call can have."""
import math

import numpy as np
import pytest

import bit_weight_only_w4_b200 as w4
from tests.gpu_util import act_order, skip_without_gpu, torch_mod
from tests.test_gpu_epilogue import Layer, check, reference

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


@pytest.mark.parametrize("activation", ["silu", "gelu_tanh", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("M", [5, 40, 300])
def test_activations_of_exact_sums_in_fp32(M, dtype, gated, activation):
    """One channel of a row is not zero, scales are a power of two: every sum x (q - 8) / 8 is exact,
    and an fp32 output is its activation alone.  With e = 2^-24: SiLU's exponential is within
    2^-22 (2^x) + 4 e, the sum and the quotient add 2^-22 + e: below 2^-20 of the value.  The GELUs'
    arguments are rounded, a relative 6 e, and their tails go as e^-u with u below 1 + x^2 (tanh: 1.6 |x|
    + 0.072 |x|^3 as far as the range here, |x| <= 12; erf: x^2 / 2): within 2^-20 (1 + x^2) of the value.
    A gated output adds one product.  Quotients by more than 2^126 are zero: |x| 2^-126."""
    skip_without_gpu()
    torch = torch_mod()
    N, K = 128, 128
    L = Layer(22, N, K, 128, True, dtype=dtype)
    L.sc.fill_(0.125)
    q = (L.what / Layer(22, N, K, 128, True, dtype=dtype).sc.double().repeat_interleave(128, 0).t()).round()
    g = torch.Generator(device="cuda").manual_seed(M)
    most = 12.0 if activation != "silu" else 80.0
    x = ((torch.rand(M, generator=g, device="cuda") * 2 - 1) * most).to(L.dt)
    X = torch.zeros(M, K, device="cuda").to(L.dt)
    at = torch.randint(0, K, (M,), generator=g, device="cuda")
    X[torch.arange(M, device="cuda"), at] = x
    t = x.double()[:, None] * q[:, at].t() / 8
    Y = w4.w4a16_gemm_epi(X, L.qw, L.sc, None, 128, activation=activation, gated=gated, out_dtype=torch.float32)
    if gated:
        t = t.view(M, -1, 2, 8)
        t, up = t[:, :, 0].reshape(M, -1), t[:, :, 1].reshape(M, -1)
    # (forms that keep the negative tails' digits: 1 + tanh and 1 + erf lose them in 64 bits too)
    want = {"silu": lambda: t * torch.sigmoid(t), "gelu": lambda: 0.5 * t * torch.erfc(-t / 2 ** 0.5),
            "gelu_tanh": lambda: t * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (t + 0.044715 * t ** 3))}[activation]()
    rel = 2.0 ** -20 * (1 if activation == "silu" else 1 + t ** 2)
    if gated:
        want = want * up
        rel = rel + 2.0 ** -24
    bad = (Y.double() - want).abs() > rel * want.abs() + 2.0 ** -126 * (1 + t.abs()) * (1 + (up.abs() if gated else 0))
    assert not bad.any(), (int(bad.sum()), t[bad][:4], Y[bad][:4], want[bad][:4])
    assert t.abs().max() > 0.5 * most


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("perm", [False, True])
@pytest.mark.parametrize("M", [33, 50, 64])
def test_two_products_strided_in_place_permuted_and_captured(M, perm, dtype):
    """33 to 64 rows, 32-channel groups, zero points: each of the two products has to find its rows
    of X, Y, the residual and the gathered columns."""
    skip_without_gpu()
    torch = torch_mod()
    K, g = 576, 32
    g_idx = act_order(np.random.default_rng(4), K, g) if perm else None
    L = Layer(23, 208, K, g, dtype=dtype, g_idx=g_idx, perm=perm)
    X = L.acts(M)
    bias = torch.randn(208, generator=L.gen, device="cuda")
    s_inv = torch.rand(K, generator=L.gen, device="cuda") + 0.5
    for gated, n_out in ((False, 208), (True, 104)):
        for out in (L.dt, torch.float32):
            wide = torch.randn(M, n_out + 96, generator=L.gen, device="cuda").to(out)
            keep = wide.clone()
            Y = wide[:, 32:32 + n_out]
            kw = dict(bias=bias, activation="silu", gated=gated, s_inv=s_inv, perm=L.perm)
            ref = reference(L, X, bias, "silu", gated, keep[:, 32:32 + n_out], s_inv)
            w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, g, residual=Y, Y=Y, **kw)     # in place, rows apart
            check(Y, ref)
            want = Y.clone()
            assert torch.equal(wide[:, :32], keep[:, :32]) and torch.equal(wide[:, 32 + n_out:], keep[:, 32 + n_out:])
            far = torch.full((M, n_out + 8), 5.0, device="cuda").to(out)          # another stride than the residual's
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, g, residual=keep[:, 32:32 + n_out], Y=far[:, :n_out], **kw)
            for _ in range(2):
                far[:, :n_out].zero_()
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(far[:, :n_out], want) and bool((far[:, n_out:] == 5).all())
    # the plain entry points: rows of the two products are rows of products alone
    whole = w4.w4a16_gemm(X, L.qw, L.sc, L.zr, g, s_inv=s_inv, perm=L.perm)
    parts = [w4.w4a16_gemm(X[a:b].contiguous(), L.qw, L.sc, L.zr, g, s_inv=s_inv, perm=L.perm) for a, b in ((0, 32), (32, M))]
    assert torch.equal(whole, torch.cat(parts))
    w4.w4_check_device_error()
