"""Rotary positions against a plain fp64 implementation.

Bound of one output a' = m (a cos phi - b sin phi): the fp64 angle is exact here (the
reference forms the same fp64 product; reducing it to turns costs 2^-52 |phi|, at most 2^-20
at position 2^31), its fraction of a turn is rounded to fp32 (2^-25 of half turns: 2^-23
radians), sine and cosine are within 2^-22, the products and the sum within 2^-22 of
|a| + |b|: together below 2^-19 m (|a| + |b|), plus the output's rounding."""
import math

import numpy as np
import pytest

import bit_weight_only_w4_b200 as w4
from tests.gpu_util import skip_without_gpu, torch_mod

pytestmark = pytest.mark.gpu


def reference(X, pos, inv, interleaved, m):
    torch = torch_mod()
    x = X.double()
    n = inv.shape[0]
    i = torch.arange(n, device=X.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    phi = (pos.double()[:, None] * inv)[:, None]
    y, e = x.clone(), torch.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = m * (a * phi.cos() - b * phi.sin())
    y[..., ib] = m * (b * phi.cos() + a * phi.sin())
    e[..., ia] = e[..., ib] = 2.0 ** -19 * abs(m) * (a.abs() + b.abs())
    return y, e


def check(Y, X, pos, inv, interleaved, m):
    torch = torch_mod()
    y, e = reference(X, pos, inv, interleaved, m)
    u = torch.finfo(Y.dtype).eps / 2
    bad = (Y.double() - y).abs() > e * 1.01 + u * y.abs() * 1.001 + torch.finfo(Y.dtype).tiny * u
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    rot = 2 * inv.shape[0]
    assert torch.equal(Y[..., rot:], X[..., rot:])


def freqs(rot, theta=10000.0):
    torch = torch_mod()
    return theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,rot", [(1, 40, 128, 128), (1, 1, 64, 64), (33, 3, 128, 64), (700, 8, 96, 96),
                                       (5, 2, 80, 32), (17, 3, 20, 6), (2, 1, 2, 2), (3, 2, 130, 130),
                                       (9, 64, 512, 512), (4, 300, 64, 16), (0, 4, 64, 64)])
def test_shapes(T, H, D, rot, interleaved, dtype):
    skip_without_gpu()
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(T + H)
    X = torch.randn(T, H, D, generator=g, device="cuda").to(getattr(torch, dtype))
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda").int()
    Y = w4.w4_rope(X, pos, freqs(rot), interleaved=interleaved, mscale=1.125)
    w4.w4_check_device_error()
    check(Y, X, pos, freqs(rot), interleaved, 1.125)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(interleaved):
    skip_without_gpu()
    torch = torch_mod()
    pos = torch.tensor([0, 1, -1, -77, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31)], device="cuda").int()
    X = torch.randn(8, 2, 64, device="cuda")
    check(w4.w4_rope(X, pos, freqs(64), interleaved=interleaved), X, pos, freqs(64), interleaved, 1.0)


@pytest.mark.parametrize("dtype", ["float16", "float32"])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("rot", [128, 48])
def test_slices_in_place_and_layouts(rot, offset, dtype):
    """The query and key heads of fused rows, in place and into a head-major buffer; rows
    that do not start on 16 bytes; what is not rotated stays."""
    skip_without_gpu()
    torch = torch_mod()
    dt = getattr(torch, dtype)
    T, H, Hk, D = 37, 4, 2, 128
    buf = torch.randn(T, (H + 2 * Hk) * D + 8 + offset, device="cuda").to(dt)
    keep = buf.clone()
    view = buf[:, offset:offset + (H + Hk) * D].unflatten(1, (H + Hk, D))
    orig = view.clone()
    pos = torch.arange(100, 100 + T, device="cuda").int()
    heads_first = torch.full((H + Hk, T, D), 7.0, device="cuda").to(dt)
    w4.w4_rope(view, pos, freqs(rot), Y=heads_first.transpose(0, 1))
    check(heads_first.transpose(0, 1), orig, pos, freqs(rot), False, 1.0)
    assert torch.equal(buf, keep)
    assert w4.w4_rope(view, pos, freqs(rot), Y=view) is view
    check(view, orig, pos, freqs(rot), False, 1.0)
    rest = torch.ones(buf.shape[1], dtype=torch.bool)
    rest[offset:offset + (H + Hk) * D] = False
    assert torch.equal(buf[:, rest], keep[:, rest])


def test_non_finite_values_stay_in_their_pair():
    skip_without_gpu()
    torch = torch_mod()
    X = torch.randn(2, 2, 64, device="cuda").half()
    X[0, 1, 3] = float("inf")
    X[1, 0, 40] = float("nan")
    Y = w4.w4_rope(X, torch.tensor([3, 4], device="cuda").int(), freqs(64))
    bad = ~Y.isfinite()
    want = torch.zeros_like(bad)
    want[0, 1, 3] = want[0, 1, 35] = want[1, 0, 8] = want[1, 0, 40] = True
    assert torch.equal(bad, want)


def test_captured_and_on_another_stream():
    skip_without_gpu()
    torch = torch_mod()
    X = torch.randn(130, 10, 128, device="cuda").bfloat16()
    pos, inv = torch.arange(130, device="cuda").int(), freqs(128)
    want = w4.w4_rope(X, pos, inv)
    Y = torch.zeros_like(X)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w4.w4_rope(X, pos, inv, Y=Y, stream=s)
    s.synchronize()
    assert torch.equal(Y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.w4_rope(X, pos, inv, Y=Y)
    pos += 5
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, w4.w4_rope(X, torch.arange(5, 135, device="cuda").int(), inv))


def test_frequencies_reach_the_kernel():
    """w4_rope_freqs' vector on the device, and a linear stretch as slower positions."""
    skip_without_gpu()
    torch = torch_mod()
    inv, m = w4.w4_rope_freqs(128, 10000.0)
    assert inv.is_cuda and m == 1.0 and np.allclose(inv.cpu().numpy(), freqs(128).cpu().numpy(), rtol=1e-14)
    inv4, _ = w4.w4_rope_freqs(128, 10000.0, "linear", factor=4.0)
    X = torch.randn(6, 2, 128, device="cuda").half()
    pos = torch.arange(6, device="cuda").int()
    assert torch.equal(w4.w4_rope(X, 4 * pos, inv4), w4.w4_rope(X, pos, inv))
    assert math.isclose(w4.w4_rope_freqs(64, scaling="ramp", factor=16.0, lo=1.0, hi=32.0)[1], 0.1 * math.log(16) + 1,
                        rel_tol=1e-6)
