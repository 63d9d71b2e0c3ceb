"""W4A16 products with an epilogue against a plain fp64 implementation.

Bound of one output.  With what = the dequantised weights, x = the activations as they reach
the product, and D the deviation of a sum t = sum_k x what + bias:
  prefill (M > 64) and fp16 decode multiply exact integers (fp16 decode: codes times 2^-24 or
  2^-20, the zero point removed with the activation sums): every partial sum is below
  A = sum_k |x| (15 + z) scale, and adding K products and K / 32 group sums in fp32, each
  addition off by at most 2^-23 of it (tensor cores truncate), keeps
      D <= (K / 8 + K / 32 + 16) 2^-23 A       (the tensor cores add at least 8 at a time)
  bf16 decode multiplies codes biased by 128: the same with (143 + 128 + z) in place of
  (15 + z).  Act-order (fp16) rounds each weight to fp16: plus 2^-11 sum |x what| twice (the
  product and the difference q - z, exact, times the scale).  s_inv rounds x: the reference
  uses the rounded x.
An activation has a slope of at most 1.13, so an output act(t) is off by 1.13 D, a gated one
by 1.13 D_gate |t_up| + |act(t_gate)| D_up + their product, plus 2^-19 of itself for the
fp32 activation (2^x within 2 ulp for arguments up to 2^4, a few more operations; beyond,
where e^-x is large, the result is below 2^-20 of the terms here), plus the output's rounding."""
import numpy as np
import pytest

import bit_weight_only_w4_b200 as w4
from tests.gpu_util import act_order, skip_without_gpu, torch_mod

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, seed, N, K, group, symmetric=False, dtype="float16", g_idx=None, perm=False):
        torch = torch_mod()
        g = torch.Generator(device="cuda").manual_seed(seed)
        W = (torch.randn(N, K, generator=g, device="cuda") * 0.02).half()
        self.g_idx = self.perm = None
        order = torch.arange(K, device="cuda")
        groups = order // group
        if g_idx is not None:
            gi = torch.from_numpy(g_idx).cuda()
            groups = gi.long()
            if perm:
                self.perm = w4.w4_actorder_perm(gi, group)
            else:
                self.g_idx = gi
        self.qw, self.sc, self.zr = w4.w4_quantize_pack(W, None, group, symmetric, g_idx=self.g_idx, perm=self.perm)
        words = w4.w4_unpack_canonical(self.qw, N, K).long() & 0xFFFFFFFF
        q = ((words[..., None] >> torch.arange(0, 32, 4, device="cuda")) & 15).reshape(N, K).double()
        if self.perm is not None:   # packed columns back in channel order
            u = torch.empty_like(q)
            u[:, self.perm.long()] = q
            q = u
        sc = self.sc.double()[groups].t()
        z = torch.full_like(sc, 8.0) if self.zr is None else self.zr.double()[groups].t()
        self.what, self.bound, self.bias_bound = (q - z) * sc, (15 + z) * sc, (271 + z) * sc
        self.N, self.K, self.group, self.dt = N, K, group, getattr(torch, dtype)
        self.gen = g

    def acts(self, M):
        torch = torch_mod()
        return torch.randn(M, self.K, generator=self.gen, device="cuda").to(self.dt)


def act64(x, name):
    torch = torch_mod()
    if name in (None, "none"):
        return x
    if name == "relu":
        return x.clamp_min(0)
    if name == "silu":
        return x * torch.sigmoid(x)
    if name == "gelu":
        return x * torch.special.ndtr(x)
    return 0.5 * x * (1 + torch.tanh((2 / np.pi) ** 0.5 * (x + 0.044715 * x ** 3)))


def reference(L, X, bias=None, activation=None, gated=False, residual=None, s_inv=None):
    """(Y, bound without the output's rounding) in fp64."""
    x = X.double()
    if s_inv is not None:
        x = (X.float() * s_inv).to(X.dtype).double()
    t = x @ L.what.t()
    M = X.shape[0]
    biased = L.dt == torch_mod().bfloat16 and M <= 64
    A = x.abs() @ (L.bias_bound if biased else L.bound).t()
    D = (L.K / 8 + L.K / 32 + 16) * 2.0 ** -23 * A
    if L.g_idx is not None:
        D = D + 2.0 ** -10 * (x.abs() @ L.what.abs().t())
    if bias is not None:
        t = t + bias.double()
        D = D + 2.0 ** -23 * t.abs()
    if gated:
        t, D = t.view(M, -1, 2, 8), D.view(M, -1, 2, 8)
        gate, up = act64(t[:, :, 0], activation), t[:, :, 1]
        dg, du = 1.13 * D[:, :, 0] + 2.0 ** -19 * gate.abs(), D[:, :, 1]
        y, e = gate * up, dg * up.abs() + gate.abs() * du + dg * du
        y, e = y.reshape(M, -1), e.reshape(M, -1)
    else:
        y = act64(t, activation)
        e = 1.13 * D + (2.0 ** -19 * y.abs() if activation else 0)
    if residual is not None:
        y = y + residual.double()
        e = e + 2.0 ** -23 * (y.abs() + residual.double().abs())
    return y, e


def check(Y, ref):
    torch = torch_mod()
    y, e = ref
    u = torch.finfo(Y.dtype).eps / 2
    tol = e * (1 + u) + u * y.abs() * 1.001 + 2.0 ** -20 * e + torch.finfo(Y.dtype).tiny * u + 1e-20
    bad = (Y.double() - y).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), Y[bad][:4], y[bad][:4], tol[bad][:4])


def run(L, M, seed=0, **kw):
    torch = torch_mod()
    X = L.acts(M)
    n_out = L.N // 2 if kw.get("gated") else L.N
    r = lambda *s, dt=L.dt: torch.randn(*s, generator=L.gen, device="cuda").to(dt)  # noqa: E731
    call = dict(kw)
    if kw.get("bias"):
        call["bias"] = r(L.N, dt=getattr(torch, kw["bias"]))
    if kw.get("residual"):
        call["residual"] = r(M, n_out, dt=getattr(torch, kw["residual"]))
    s_inv = None
    if kw.get("s_inv"):
        call["s_inv"] = s_inv = torch.rand(L.K, generator=L.gen, device="cuda") + 0.5
    if kw.get("out_dtype"):
        call["out_dtype"] = getattr(torch, kw["out_dtype"])
    Y = w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, L.group, g_idx=L.g_idx, perm=L.perm, **call)
    w4.w4_check_device_error()
    ref = reference(L, X, call.get("bias"), kw.get("activation"), kw.get("gated", False), call.get("residual"), s_inv)
    check(Y, ref)
    return X, Y, call


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("M", [1, 3, 8, 9, 16, 17, 32, 40, 64, 65, 256, 257, 300])
def test_every_batch_size(M, dtype):
    """One layer of two bands (the last one ragged) whose bands are split between CTAs, with
    bias, SiLU and residual."""
    skip_without_gpu()
    L = Layer(M, 208, 2048, 128, dtype=dtype)
    run(L, M, bias=dtype, activation="silu", residual=dtype)
    run(L, M, activation="silu", gated=True, residual=dtype)


@pytest.mark.parametrize("activation", [None, "none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [2, 70])
def test_activations(M, gated, activation):
    skip_without_gpu()
    L = Layer(5, 144, 512, 64)
    run(L, M, activation=activation, gated=gated, bias="float32")


@pytest.mark.parametrize("out_dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("residual", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("M", [5, 100])
def test_types(M, residual, out_dtype):
    skip_without_gpu()
    L = Layer(6, 256, 256, 32, symmetric=True, dtype="bfloat16")
    run(L, M, activation="relu", residual=residual, out_dtype=out_dtype, bias="bfloat16")
    run(L, M, activation="gelu", gated=True, residual=residual, out_dtype=out_dtype, bias="float16")


@pytest.mark.parametrize("group,K", [(32, 320), (64, 448), (192, 384), (128, 640), (1024, 1024)])
@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("M", [4, 12, 130])
def test_groups(M, symmetric, group, K):
    skip_without_gpu()
    for dtype in ("float16", "bfloat16"):
        L = Layer(7, 96, K, group, symmetric, dtype)
        run(L, M, activation="silu", gated=True, bias=dtype, s_inv=True)
        run(L, M, residual=dtype)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("M", [33, 47, 64])
def test_small_groups_with_zero_points_between_33_and_64_rows(M, dtype):
    """Where one stage would not fit shared memory twice the rows are done in two parts; the
    plain product the same."""
    skip_without_gpu()
    torch = torch_mod()
    L = Layer(13, 144, 576, 32, dtype=dtype)
    run(L, M, bias=dtype, activation="silu", residual="float32")
    run(L, M, activation="gelu", gated=True, residual=dtype, s_inv=True)
    X = L.acts(M)
    Y = w4.w4a16_gemm(X, L.qw, L.sc, L.zr, 32, out_dtype=torch.float32)
    y, e = reference(L, X)
    biased = (L.K / 8 + L.K / 32 + 16) * 2.0 ** -23 * (X.double().abs() @ (L.bound + 1024 * L.sc.double().repeat_interleave(32, 0).t()).t())
    assert ((Y.double() - y).abs() <= e + 16 * biased).all()   # (the plain product's fp16 codes are biased by 1024, rows r + 8 by 64 of 16 q)


@pytest.mark.parametrize("perm", [False, True])
@pytest.mark.parametrize("M", [1, 20, 80])
def test_act_order(M, perm):
    skip_without_gpu()
    K, g = 512, 64
    L = Layer(8, 160, K, g, True, g_idx=act_order(np.random.default_rng(3), K, g), perm=perm)
    run(L, M, activation="gelu_tanh", bias="float16", residual="float16")
    run(L, M, activation="silu", gated=True)


@pytest.mark.parametrize("M", [1, 33, 128])
def test_residual_in_place_and_row_strides(M):
    """The residual may be Y itself; Y and the residual may be column slices; what lies
    between the slices' rows stays."""
    skip_without_gpu()
    torch = torch_mod()
    L = Layer(9, 192, 512, 128)
    X = L.acts(M)
    wide = torch.randn(M, 400, generator=L.gen, device="cuda").half()
    keep = wide.clone()
    Y = wide[:, 96:96 + 192]
    out = w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, 128, activation="silu", residual=Y, Y=Y)
    assert out is Y
    check(Y, reference(L, X, activation="silu", residual=keep[:, 96:288]))
    assert torch.equal(wide[:, :96], keep[:, :96]) and torch.equal(wide[:, 288:], keep[:, 288:])


def test_empty_batch_and_nan():
    skip_without_gpu()
    torch = torch_mod()
    L = Layer(10, 128, 256, 128)
    assert w4.w4a16_gemm_epi(L.acts(0), L.qw, L.sc, L.zr, 128, activation="silu").shape == (0, 128)
    for M in (2, 90):   # a NaN or infinite activation reaches its own row alone, also through ReLU
        X = L.acts(M)
        X[1, 5] = float("nan")
        Y = w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, 128, activation="relu")
        assert Y[1].isnan().all() and Y[0].isfinite().all()


def test_plain_product_is_unchanged_by_an_epilogue_call_between():
    """Both entry points share one workspace on a stream and leave it ready for each other."""
    skip_without_gpu()
    torch = torch_mod()
    L = Layer(11, 1024, 4096, 128)
    for M in (1, 16, 64, 200):
        X = L.acts(M)
        first = w4.w4a16_gemm(X, L.qw, L.sc, L.zr, 128)
        for _ in range(3):
            w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, 128, activation="silu", gated=True)
        assert torch.equal(w4.w4a16_gemm(X, L.qw, L.sc, L.zr, 128), first)


def test_captured_and_on_another_stream():
    skip_without_gpu()
    torch = torch_mod()
    L = Layer(12, 512, 2048, 128)
    for M in (1, 24, 96):
        X = L.acts(M)
        need = max(w4.w4a16_workspace_bytes(M, L.N, L.K, 128), 256)
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        want = w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, 128, activation="silu", gated=True)
        Y = torch.zeros_like(want)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, 128, activation="silu", gated=True, Y=Y, workspace=ws, stream=s)
        s.synchronize()
        assert torch.equal(Y, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, 128, activation="silu", gated=True, Y=Y, workspace=ws)
        for _ in range(3):
            Y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(Y, want)
        X.copy_(L.acts(M))   # a replay reads the buffers as they are then
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, 128, activation="silu", gated=True))


def test_gated_rows():
    skip_without_gpu()
    torch = torch_mod()
    F, K = 24, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    gate, up = (torch.randn(F, K, generator=g, device="cuda").half() * 0.05 for _ in range(2))
    order = w4.gated_rows(F, "cuda")
    qw, sc, zr = w4.w4_quantize_pack(torch.cat([gate, up])[order].contiguous(), None, 128)
    X = torch.randn(3, K, generator=g, device="cuda").half()
    t = w4.w4a16_gemm(X, qw, sc, zr, 128, out_dtype=torch.float32).double()
    both = torch.empty_like(t)
    both[:, order] = t           # rows of [gate; up] again
    want = act64(both[:, :F], "silu") * both[:, F:]
    got = w4.w4a16_gemm_epi(X, qw, sc, zr, 128, activation="silu", gated=True, out_dtype=torch.float32).double()
    # the plain product's own fp32 error (biased codes) against the epilogue's: 2^-23 K/8 terms of 1024 |x| scale
    assert torch.allclose(got, want, rtol=0, atol=float(16 * 2.0 ** -23 * 1040 * X.double().abs().sum(1).max()
                                                       * sc.double().max() * (1 + t.abs().max()) * 2.3))
