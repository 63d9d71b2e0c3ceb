"""Host side of the product with an epilogue, the rotary positions and prompt attention:
refusals of the C entry points and of the binding (nothing here reaches a GPU), and the
rotary frequencies, which are computed on the host."""
import ctypes
import math

import numpy as np
import pytest

import bit_weight_only_w4_b200 as w4
from bit_weight_only_w4_b200 import build

P = 1 << 20   # an aligned address that no refused call dereferences


@pytest.fixture(scope="module")
def L():
    build.build()
    return w4.lib()


# ---------------------------------------------------------------- product with an epilogue
def epi_call(L, M=1, N=128, K=128, g=128, out=0, g_idx=None, perm=None, null=False, ws=P, **kw):
    e = w4.Epilogue()
    for k, v in kw.items():
        setattr(e, k, v)
    return L.w4a16_gemm_epi(P, 0, M, N, K, P, P, None, g_idx, perm, g, None, None if null else ctypes.byref(e), P, out, ws,
                            1 << 40, None)


def test_epilogue_refusals(L):
    bad = w4.W4_ERR_INVALID_ARG
    assert epi_call(L, null=True) == bad
    assert epi_call(L, g_idx=P, perm=P) == bad
    assert epi_call(L, activation=5) == bad and epi_call(L, activation=-1) == bad
    assert epi_call(L, gated=2) == bad
    assert epi_call(L, out=3) == bad
    assert epi_call(L, bias=P, bias_dtype=3) == bad and epi_call(L, bias=P + 1) == bad
    assert epi_call(L, bias=P + 2, bias_dtype=2) == bad
    assert epi_call(L, residual=P, residual_dtype=7) == bad and epi_call(L, residual=P + 8) == bad
    assert epi_call(L, ldy=120) == bad and epi_call(L, ldy=129) == bad and epi_call(L, ldy=-128) == bad
    assert epi_call(L, residual=P + 16, ldr=64) == bad and epi_call(L, residual=P + 16, ldr=132) == bad
    assert epi_call(L, gated=1, ldy=56) == bad
    # the residual is Y: only with Y's rows and type
    assert epi_call(L, residual=P, ldr=256) == bad
    assert epi_call(L, residual=P, residual_dtype=2) == bad
    # as w4a16_gemm
    assert epi_call(L, N=8) == w4.W4_ERR_UNSUPPORTED and epi_call(L, K=96, g=32) == w4.W4_ERR_UNSUPPORTED
    assert epi_call(L, M=-1) == bad
    assert epi_call(L, M=0) == w4.W4_OK


def test_epilogue_binding_refusals():
    import torch
    N, K, g = 32, 64, 64
    X = torch.zeros(2, K, dtype=torch.float16)
    qw, sc = torch.zeros(N * K // 8, dtype=torch.int32), torch.zeros(1, N, dtype=torch.float16)
    call = lambda **kw: w4.w4a16_gemm_epi(X, qw, sc, sc, g, **kw)  # noqa: E731
    with pytest.raises(ValueError, match="activation"):
        call(activation="tanh")
    with pytest.raises(ValueError, match="bias"):
        call(bias=torch.zeros(N - 1))
    with pytest.raises(TypeError, match="bias"):
        call(bias=torch.zeros(N, dtype=torch.float64))
    with pytest.raises(ValueError, match="g_idx or perm"):
        call(g_idx=torch.zeros(K, dtype=torch.int32), perm=torch.zeros(K, dtype=torch.int32))
    with pytest.raises(ValueError, match="qweight"):
        w4.w4a16_gemm_epi(X, qw[:-1], sc, sc, g)
    with pytest.raises(ValueError, match="CUDA"):
        call(activation="silu", gated=True)


def test_gated_rows_order():
    assert w4.gated_rows(16).tolist() == list(range(8)) + list(range(16, 24)) + list(range(8, 16)) + list(range(24, 32))
    with pytest.raises(ValueError):
        w4.gated_rows(12)


# ---------------------------------------------------------------- rotary positions
def rope_call(L, X=P, dtype=0, T=4, H=2, D=64, sx=(128, 64), pos=P, inv=P, rot=64, m=1.0, inter=0, Y=2 * P, sy=(128, 64)):
    return L.w4_rope(X, dtype, T, H, D, sx[0], sx[1], pos, inv, rot, m, inter, Y, sy[0], sy[1], None)


def test_rope_refusals(L):
    bad = w4.W4_ERR_INVALID_ARG
    assert rope_call(L, dtype=3) == bad and rope_call(L, T=-1) == bad and rope_call(L, H=-1) == bad
    assert rope_call(L, D=0) == bad
    for rot in (0, 1, 63, 66, -2):
        assert rope_call(L, rot=rot) == bad, rot
    assert rope_call(L, D=1024, rot=514, sx=(2048, 1024), sy=(2048, 1024)) == w4.W4_ERR_UNSUPPORTED
    assert rope_call(L, inter=2) == bad
    assert rope_call(L, m=float("nan")) == bad and rope_call(L, m=float("inf")) == bad
    for n in ("X", "Y", "pos", "inv"):
        assert rope_call(L, **{n: None}) == bad, n
    assert rope_call(L, X=P + 1) == bad and rope_call(L, inv=P + 4) == bad and rope_call(L, pos=P + 2) == bad
    assert rope_call(L, dtype=2, Y=P + 2) == bad
    assert rope_call(L, sy=(128, 32)) == bad and rope_call(L, sy=(32, 64)) == bad   # outputs that overlap
    assert rope_call(L, sx=(-128, 64)) == bad
    assert rope_call(L, Y=P, sy=(256, 64)) == bad                                   # in place: equal strides
    assert rope_call(L, T=0) == w4.W4_OK and rope_call(L, H=0, X=None, Y=None) == w4.W4_OK


def shared_places(T, H, D, st, sh):
    """Whether two elements of a [T, H, D] view with these strides share a place."""
    at = (np.arange(T)[:, None, None] * st + np.arange(H)[None, :, None] * sh + np.arange(D)).ravel()
    return len(np.unique(at)) < at.size


def test_rope_refuses_outputs_that_share_elements(L):
    """Every pair of strides of small views, among them those where each stride alone leaves
    room for a head; the accepted ones are told by the missing device (this test's pointers are
    no memory, and accepted calls end at the device query)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("accepted calls would be launched")
    D = 4
    for T, H in ((2, 2), (3, 2), (2, 5), (4, 3), (7, 6)):
        for st in range(0, 40):
            for sh in range(0, 40):
                got = rope_call(L, T=T, H=H, D=D, rot=D, sx=(H * D, D), sy=(st, sh))
                want = w4.W4_ERR_INVALID_ARG if shared_places(T, H, D, st, sh) else w4.W4_ERR_CUDA
                assert got == want, (T, H, st, sh, got)
    big = 1 << 61   # products of strides and counts pass 64 bits
    assert rope_call(L, T=1 << 20, H=1 << 15, sy=(64, big)) == w4.W4_ERR_CUDA
    assert rope_call(L, T=1 << 20, H=1 << 15, sy=(64, 64 << 19)) == w4.W4_ERR_INVALID_ARG


def freqs(rot, theta=10000.0, scaling=0, factor=1.0, context=8192.0, lo=1.0, hi=4.0):
    out, m = (ctypes.c_double * max(1, rot // 2))(), ctypes.c_float()
    st = w4.lib().w4_rope_freqs(rot, theta, scaling, factor, context, lo, hi, out, ctypes.byref(m))
    return st, np.array(out[:]), m.value


@pytest.mark.parametrize("rot,theta", [(2, 10000.0), (64, 10000.0), (128, 500000.0)])
def test_rope_freqs_plain_linear_base(L, rot, theta):
    i = np.arange(rot // 2)
    st, f, m = freqs(rot, theta)
    assert st == w4.W4_OK and m == 1.0 and np.allclose(f, theta ** (-2.0 * i / rot), rtol=1e-14)
    assert np.allclose(freqs(rot, theta, w4.W4_ROPE_LINEAR, 8.0)[1], f / 8.0, rtol=1e-14)
    if rot > 2:
        st, g, m = freqs(rot, theta, w4.W4_ROPE_BASE, 8.0)
        assert g[0] == 1.0 and math.isclose(g[-1], f[-1] / 8.0, rel_tol=1e-12)   # the slowest pair stretches by the factor


def test_rope_freqs_bands(L):
    _, f, _ = freqs(128, 500000.0)
    st, g, m = freqs(128, 500000.0, w4.W4_ROPE_BANDS, 8.0, 8192.0, 1.0, 4.0)
    assert st == w4.W4_OK and m == 1.0
    for a, b in zip(f, g):
        w = 2 * math.pi / a
        if w < 8192 / 4:
            want = a
        elif w > 8192:
            want = a / 8
        else:
            s = (8192 / w - 1) / 3
            want = (1 - s) * a / 8 + s * a
        assert math.isclose(b, want, rel_tol=1e-12)
    assert g[0] == f[0] and math.isclose(g[-1], f[-1] / 8)


def test_rope_freqs_ramp(L):
    rot, theta, ctx = 128, 10000.0, 4096.0
    _, f, _ = freqs(rot, theta)
    st, g, m = freqs(rot, theta, w4.W4_ROPE_RAMP, 16.0, ctx, 1.0, 32.0)
    assert st == w4.W4_OK and math.isclose(m, 0.1 * math.log(16) + 1, rel_tol=1e-6)
    at = lambda r: rot * math.log(ctx / (r * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    first, last = max(math.floor(at(32)), 0), min(math.ceil(at(1)), rot - 1)
    r = np.clip((np.arange(rot // 2) - first) / (last - first), 0, 1)
    assert np.allclose(g, f * (1 - r) + f / 16 * r, rtol=1e-12)
    assert freqs(rot, theta, w4.W4_ROPE_RAMP, 0.5, ctx, 1.0, 32.0)[2] == 1.0


def test_rope_freqs_refusals(L):
    bad = w4.W4_ERR_INVALID_ARG
    for kw in (dict(rot=0), dict(rot=7), dict(rot=514), dict(rot=64, theta=1.0), dict(rot=64, theta=float("nan")),
               dict(rot=64, scaling=5), dict(rot=64, scaling=1, factor=0.0), dict(rot=64, scaling=1, factor=float("inf")),
               dict(rot=2, scaling=2, factor=2.0), dict(rot=64, scaling=3, factor=2.0, context=0.0),
               dict(rot=64, scaling=3, factor=2.0, lo=4.0, hi=4.0), dict(rot=64, scaling=4, factor=2.0, lo=0.0)):
        assert freqs(**kw)[0] == bad, kw
    assert L.w4_rope_freqs(64, 10000.0, 0, 1.0, 1.0, 1.0, 2.0, None, None) == bad
    with pytest.raises(ValueError, match="scaling"):
        w4.w4_rope_freqs(64, scaling="cubic", device="cpu")
    inv, m = w4.w4_rope_freqs(64, device="cpu")
    assert inv.shape == (32,) and str(inv.dtype) == "torch.float64" and m == 1.0


def test_rope_binding_refusals():
    import torch
    X = torch.zeros(2, 1, 8, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        w4.w4_rope(X, torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError, match="heads"):
        w4.w4_rope(X[:, 0], torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.float64))


# ---------------------------------------------------------------- prompt attention
def attn_call(L, dtype=0, ws=None, ws_bytes=0, null=False, **kw):
    a = w4.Attention(P, P, P, P, None, P, None, 16, 16, 256, 64, 256, 64, 256, 64, 256, 64, 2, 4, 4, 64, 0.125, 1)
    for k, v in kw.items():
        setattr(a, k, v)
    return L.w4_prompt_attention(None if null else ctypes.byref(a), dtype, ws, ws_bytes, None)


def test_attention_refusals(L):
    bad, un = w4.W4_ERR_INVALID_ARG, w4.W4_ERR_UNSUPPORTED
    assert attn_call(L, null=True) == bad
    assert attn_call(L, dtype=2) == bad
    for kw in (dict(batch=-1), dict(heads=0), dict(kv_heads=0), dict(kv_heads=3), dict(head_dim=0), dict(q_tokens=-1),
               dict(k_tokens=-1), dict(causal=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(cu_seqlens_q=None), dict(cu_seqlens_q=None, cu_seqlens_k=P, batch=1),
               dict(k_tokens=17), dict(Q=None), dict(K=None), dict(V=None), dict(O=None), dict(Q=P + 8), dict(O=P + 2),
               dict(lse=P + 2), dict(cu_seqlens_q=P + 2), dict(q_token_stride=32), dict(k_token_stride=260),
               dict(v_head_stride=60), dict(o_head_stride=0), dict(k_token_stride=-256)):
        assert attn_call(L, **kw) == bad, kw
    for kw in (dict(head_dim=12), dict(head_dim=136), dict(heads=516, kv_heads=4), dict(q_tokens=1 << 31),
               dict(q_token_stride=1 << 38)):
        assert attn_call(L, **kw) == un, kw
    assert attn_call(L, q_tokens=0, k_tokens=0) == w4.W4_OK
    assert attn_call(L, batch=0) == w4.W4_OK


def test_attention_workspace_bytes_of_invalid_sizes(L):
    f = w4.w4_prompt_attention_workspace_bytes
    assert f(1, 4, 3, 64, 16, 16) == 0 and f(1, 4, 4, 200, 16, 16) == 0 and f(-1, 4, 4, 64, 16, 16) == 0


def test_attention_binding_refusals():
    import torch
    t = torch.zeros(4, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        w4.w4_prompt_attention(t, t, t)
    with pytest.raises(ValueError, match="Q must be"):
        w4.w4_prompt_attention(t[0], t, t)


def test_attention_refuses_outputs_that_share_elements(L):
    """As for the rotary positions; strides are multiples of 8."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("accepted calls would be launched")
    D = 16
    for T, H in ((2, 2), (3, 2), (2, 5), (4, 3)):
        for st in range(0, 160, 8):
            for sh in range(0, 160, 8):
                got = attn_call(L, q_tokens=T, k_tokens=T, heads=H, kv_heads=H, head_dim=D, q_token_stride=H * D, q_head_stride=D,
                                k_token_stride=H * D, k_head_stride=D, v_token_stride=H * D, v_head_stride=D,
                                o_token_stride=st, o_head_stride=sh)
                want = w4.W4_ERR_INVALID_ARG if shared_places(T, H, D, st, sh) else w4.W4_ERR_CUDA
                assert got == want, (T, H, st, sh, got)


def test_attention_refuses_a_workspace_that_counts_more_than_it_holds(monkeypatch):
    """An expanded tensor has the bytes asked for by its count and one by its memory."""
    import torch
    monkeypatch.setattr(w4, "_cuda_index", lambda *t: 0)
    t = torch.zeros(4, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="contiguous"):
        w4.w4_prompt_attention(t, t, t, workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 24))


def test_attention_refuses_heads_without_elements(L, monkeypatch):
    import torch
    monkeypatch.setattr(w4, "_cuda_index", lambda *t: 0)
    monkeypatch.setattr(w4, "_on_device", lambda index, fn, *a: fn(*a))
    t = torch.zeros(4, 2, 0, dtype=torch.float16)
    with pytest.raises(w4.W4Error) as e:
        w4.w4_prompt_attention(t, t, t, workspace=torch.zeros(1, dtype=torch.uint8), stream=type("S", (), {"cuda_stream": 0}), O=t)
    assert e.value.status == w4.W4_ERR_INVALID_ARG


# ---------------------------------------------------------------- build
def test_new_kernels_do_not_spill(L):
    """The one-, four- and eight-token-tile products with an epilogue and the prompt kernels
    keep everything in registers (two token tiles run at a 96-register cap: at most 24 bytes)."""
    import os
    import re
    name, seen = None, {}
    for line in open(os.path.join(os.path.dirname(w4.LIB_PATH), "build.log")):
        m = re.search(r"Compiling entry function '([^']+)'", line)
        name = m.group(1) if m else name
        m = re.search(r"(\d+) bytes spill stores, (\d+) bytes spill loads", line)
        if m and name and re.search("epi_kernel|rope_kernel|attention", name):
            seen[name] = int(m.group(1)) + int(m.group(2))
    assert any("prefill_epi" in n for n in seen) and any("attention" in n for n in seen)
    for n, b in seen.items():
        assert b <= (48 if "decode_epi_kernelILi2E" in n else 0), (n, b)
