"""Prompt attention against a plain fp64 implementation.

Bound of one output element: with A = sum_j p_j |V_j| (p the exact weights),
  u |O|            the output's rounding (u: half a step of the type)
  u A              the weights' rounding to the input type before their product with V
  2 d A            the weights' relative error d from the scores: a score is a sum of D
                   products in fp32, off by at most D 2^-23 sum |q k| scale (each addition
                   truncates at worst), plus 2^-21 for the exponent's own fp32 arithmetic on
                   values up to 2^2..2^7 and the hardware's 2^x; twice, as the weights are
                   divided by their sum
  (nk 2^-23) A     the fp32 sums over the keys
and lse within d + nk 2^-23 + 2^-22 |lse|."""
import math

import pytest

import bit_weight_only_w4_b200 as w4
from tests.gpu_util import skip_without_gpu, torch_mod

pytestmark = pytest.mark.gpu


def make(seed, q_lens, k_lens, H, Hk, D, dtype, spread=1.0):
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: (torch.randn(*s, generator=g, device="cuda") * spread).to(dtype)  # noqa: E731
    cu = lambda n: torch.tensor([0] + list(n), device="cuda").cumsum(0).int()  # noqa: E731
    Tq, Tk = sum(q_lens), sum(k_lens)
    return r(Tq, H, D), r(Tk, Hk, D), r(Tk, Hk, D), cu(q_lens), cu(k_lens)


def plain(Q, K, V, q_lens, k_lens, causal, scale):
    """(O, lse, A, score error d) in fp64."""
    torch = torch_mod()
    Tq, H, D = Q.shape
    G = H // K.shape[1]
    O = torch.zeros(Tq, H, D, dtype=torch.float64, device=Q.device)
    A = torch.zeros_like(O)
    lse = torch.full((Tq, H), -math.inf, dtype=torch.float64, device=Q.device)
    d = torch.zeros(Tq, H, dtype=torch.float64, device=Q.device)
    a = b = 0
    for n, m in zip(q_lens, k_lens):
        i = torch.arange(n, device=Q.device)[:, None]
        j = torch.arange(m, device=Q.device)[None, :]
        seen = (j <= i + m - n) if causal else torch.ones(n, m, dtype=torch.bool, device=Q.device)
        for h in range(H):
            if n == 0 or m == 0:
                continue
            q, k, v = Q[a:a + n, h].double(), K[b:b + m, h // G].double(), V[b:b + m, h // G].double()
            s = torch.where(seen, q @ k.t() * scale, -math.inf)
            lse[a:a + n, h] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[a:a + n, h, None].clamp_min(-1e300))
            p = torch.where(seen, p, 0.0)
            O[a:a + n, h] = p @ v
            A[a:a + n, h] = p @ v.abs()
            err = (q.abs() @ k.abs().t() * scale) * (D * 2.0 ** -23)
            d[a:a + n, h] = torch.where(seen, err, 0.0).amax(1) + 2.0 ** -21 * (1 + s.masked_fill(~seen, 0).abs().amax(1))
        a, b = a + n, b + m
    return O, lse, A, d


def check(O, lse, ref, dtype, longest):
    torch = torch_mod()
    Or, lr, A, d = ref
    u = torch.finfo(dtype).eps / 2
    tol = u * Or.abs() + (u + 2 * d[..., None] + longest * 2.0 ** -23) * A + 1e-30
    tol = tol * 1.001 + torch.finfo(dtype).tiny * u
    bad = (O.double() - Or).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), O[bad][:4], Or[bad][:4], tol[bad][:4])
    empty = torch.isinf(lr)
    assert torch.equal(torch.isneginf(lse), empty)
    off = (lse.double() - lr).abs()[~empty]
    assert (off <= (d + longest * 2.0 ** -23 + 2.0 ** -22 * lr.abs() + 2.0 ** -22)[~empty]).all(), off.max()


CASES = [
    # q_lens, k_lens (None: the same), H, Hk, D
    ([1], None, 1, 1, 128),
    ([128], None, 2, 1, 128),
    ([61], None, 4, 4, 128),
    ([300], None, 8, 2, 128),
    ([513], None, 7, 1, 128),                 # rows of a tile that hold no token
    ([129, 1, 0, 255, 17], None, 6, 2, 128),
    ([1, 1, 1], [700, 1, 129], 8, 1, 128),
    ([5, 3], [133, 640], 4, 2, 64),
    ([40], [13], 4, 4, 64),                   # the first rows see no key
    ([9, 4], [0, 5], 4, 2, 80),
    ([260], None, 3, 3, 80),
    ([200, 77], None, 4, 1, 8),
    ([130], None, 128, 1, 64),                # 128 heads to a key head
    ([1000], None, 4, 2, 96),
    # one tile a sequence over several key blocks (ranges), with sequences that see nothing
    ([1, 0, 1, 1, 1], [4000, 300, 0, 1, 129], 16, 2, 128),
    ([1], [9000], 8, 8, 64),
    ([3, 16, 1], [16, 5000, 2000], 8, 1, 128),
    ([1] * 40, [7 * i for i in range(40)], 4, 1, 128),          # more than 32 sequences
    # few tiles over many keys (ranges over causal tiles)
    ([100], [3000], 2, 2, 128),
    ([260, 40], [2000, 41], 3, 1, 96),
    # more than 32 prompts, longest first; one and two tiles an item
    ([(37 * i) % 190 for i in range(45)], None, 4, 2, 64),
    ([300] * 34, None, 8, 2, 128),
    ([1 + i % 3 for i in range(150)], None, 2, 1, 64),          # one item a sequence
    ([1] * 100, [200 + 3 * i for i in range(100)], 4, 2, 64),   # ranges over more than 32 sequences
    ([5], [2], 1, 1, 16),
]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_plain(case, causal, dtype):
    skip_without_gpu()
    torch = torch_mod()
    q_lens, k_lens, H, Hk, D = CASES[case]
    same = k_lens is None
    k_lens = q_lens if same else k_lens
    dt = getattr(torch, dtype)
    Q, K, V, cu_q, cu_k = make(case, q_lens, k_lens, H, Hk, D, dt)
    O, lse = w4.w4_prompt_attention(Q, K, V, cu_q, None if same else cu_k, causal=causal, return_lse=True)
    w4.w4_check_device_error()
    check(O, lse, plain(Q, K, V, q_lens, k_lens, causal, D ** -0.5), dt, max(k_lens))


@pytest.mark.parametrize("causal", [True, False])
def test_default_is_one_sequence(causal):
    skip_without_gpu()
    torch = torch_mod()
    for n, m in ((150, 150), (7, 900)):
        Q, K, V, _, _ = make(1, [n], [m], 4, 2, 64, torch.float16)
        O, lse = w4.w4_prompt_attention(Q, K, V, causal=causal, scale=0.25, return_lse=True)
        check(O, lse, plain(Q, K, V, [n], [m], causal, 0.25), torch.float16, m)


# lengths for which a call works by items (pairs, single tiles) and by ranges
WAYS = {"pairs": ([700, 300, 500], None, 32, 8), "tiles": ([150, 60], None, 8, 2), "ranges": ([1, 2, 1], [900, 500, 130], 8, 2)}


def way(name, D=128, dtype="bfloat16", seed=5):
    torch = torch_mod()
    q, k, H, Hk = WAYS[name]
    return (q, q if k is None else k) + make(seed, q, q if k is None else k, H, Hk, D, getattr(torch, dtype))


def call(w, **kw):
    q, k, Q, K, V, cu_q, cu_k = w
    return w4.w4_prompt_attention(Q, K, V, cu_q, None if q is k else cu_k, **kw)


@pytest.mark.parametrize("name", WAYS)
def test_slices_and_layouts(name):
    """Q, K and V as slices of fused rows, O head-major in a wider buffer, and without lse."""
    skip_without_gpu()
    torch = torch_mod()
    w = way(name)
    q, k, Q, K, V, cu_q, cu_k = w
    want = call(w)
    Tq, H, D = Q.shape
    Tk, Hk, _ = K.shape
    kv = torch.cat([K, V], 1)                                     # rows of K and V heads
    Qh = Q.transpose(0, 1).contiguous().transpose(0, 1)           # head-major
    out = torch.full((H, Tq, D + 24), 3.0, device="cuda").bfloat16()
    O = out[:, :, 8:8 + D].transpose(0, 1)
    got = w4.w4_prompt_attention(Qh, kv[:, :Hk], kv[:, Hk:], cu_q, None if q is k else cu_k, O=O)
    assert got is O and torch.equal(O, want)
    assert (out[:, :, :8] == 3).all() and (out[:, :, 8 + D:] == 3).all()


@pytest.mark.parametrize("name", WAYS)
def test_rows_behind_the_last_sequence_stay(name):
    skip_without_gpu()
    torch = torch_mod()
    w = way(name)
    q, k, Q, K, V, cu_q, cu_k = w
    want = call(w)
    pad = lambda t, v: torch.cat([t, torch.full((70,) + t.shape[1:], v, device="cuda").to(t.dtype)])  # noqa: E731
    O = pad(torch.zeros_like(Q), 9.0)
    w4.w4_prompt_attention(pad(Q, float("nan")), pad(K, float("nan")), pad(V, float("inf")), cu_q, None if q is k else cu_k, O=O)
    assert (O[-70:] == 9).all()
    u = torch.finfo(torch.bfloat16).eps
    assert torch.allclose(O[:-70].float(), want.float(), rtol=u, atol=u * 0.05)   # (the padding may change the way of working)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("name", WAYS)
def test_non_finite_values_reach_only_the_rows_that_see_them(name, dtype):
    """Infinite and NaN keys and values at positions that later rows see: earlier rows and
    other sequences are untouched, rows that see them become what IEEE arithmetic gives."""
    skip_without_gpu()
    torch = torch_mod()
    w = way(name, dtype=dtype)
    q, k, Q, K, V, cu_q, cu_k = w
    clean, lse0 = call(w, return_lse=True)
    for kind in ("v inf", "v nan", "k nan"):
        V2, K2 = V.clone(), K.clone()
        hits = []
        for b in range(len(q)):
            at = k[b] - 1 - (b % 2)      # the last or last but one key of each sequence
            pos = int(cu_k[b]) + at
            if kind == "v inf":
                V2[pos, 0, 3] = float("inf")
            elif kind == "v nan":
                V2[pos, 0, 3] = float("nan")
            else:
                K2[pos, 0, 7] = float("nan")
            first = max(0, q[b] - 1 - (b % 2))   # first query that sees it
            hits.append((int(cu_q[b]) + first, int(cu_q[b + 1])))
        O, lse = w4.w4_prompt_attention(Q, K2, V2, cu_q, None if q is k else cu_k, return_lse=True)
        G = Q.shape[1] // K.shape[1]
        want = clean.float()
        for a, e in hits:
            if kind == "k nan":
                want[a:e, :G] = float("nan")
            else:
                want[a:e, :G, 3] = float("inf") if kind == "v inf" else float("nan")
        assert torch.equal(torch.isnan(O.float()), torch.isnan(want)) and torch.equal(torch.isinf(O), torch.isinf(want)), kind
        ok = want.isfinite()
        assert torch.equal(O.float()[ok], want[ok]), kind
        if kind != "k nan":
            assert torch.equal(lse, lse0)


@pytest.mark.parametrize("name", WAYS)
@pytest.mark.parametrize("spread", [30.0, 0.01])
def test_large_and_small_scores(name, spread):
    """Scores of hundreds (one key takes all; the running maximum rises again and again) and
    scores that hardly differ."""
    skip_without_gpu()
    torch = torch_mod()
    q, k, H, Hk = WAYS[name]
    k = q if k is None else k
    Q, K, V, cu_q, cu_k = make(11, q, k, H, Hk, 64, torch.float16)
    Q = (Q * spread).half()
    # rising scores: later keys point ever more along the queries' mean
    K = (K + 0.01 * torch.arange(K.shape[0], device="cuda")[:, None, None] * Q.float().mean(0, keepdim=True)[:, :Hk]).half()
    O, lse = w4.w4_prompt_attention(Q, K, V, cu_q, None if q is k else cu_k, return_lse=True)
    check(O, lse, plain(Q, K, V, q, k, True, 0.125), torch.float16, max(k))


@pytest.mark.parametrize("name", WAYS)
def test_captured_and_on_another_stream(name):
    skip_without_gpu()
    torch = torch_mod()
    w = way(name)
    want, lse = call(w, return_lse=True)
    O = torch.zeros_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(w, O=O, stream=s)
    s.synchronize()
    assert torch.equal(O, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(w, O=O)
    for _ in range(2):
        O.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, want)
    # two calls at once on two streams
    s2 = torch.cuda.Stream()
    O2 = torch.zeros_like(want)
    s.wait_stream(torch.cuda.current_stream())
    s2.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        call(w, O=O, stream=s)
        call(w, O=O2, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(O, want) and torch.equal(O2, want)
    w4.w4_check_device_error()


def test_lengths_may_change_between_replays():
    """The bounds are read on the GPU: a captured call serves other lengths of the same totals."""
    skip_without_gpu()
    torch = torch_mod()
    Q, K, V, cu_q, cu_k = make(3, [100, 200, 30], [100, 200, 30], 4, 2, 64, torch.float16)
    O = torch.zeros_like(Q)
    graph = torch.cuda.CUDAGraph()
    w4.w4_prompt_attention(Q, K, V, cu_q, O=O)
    with torch.cuda.graph(graph):
        w4.w4_prompt_attention(Q, K, V, cu_q, O=O)
    cu_q.copy_(torch.tensor([0, 7, 290, 330], device="cuda").int())
    graph.replay()
    torch.cuda.synchronize()
    lens = [7, 283, 40]
    ref = plain(Q, K, V, lens, lens, True, 0.125)
    _, lse = w4.w4_prompt_attention(Q, K, V, cu_q, return_lse=True)
    check(O, lse, ref, torch.float16, 283)


@pytest.mark.parametrize("bounds", [[0, 50, 40, 100], [-5, 20, 60, 100], [0, 30, 99, 5000]])
def test_bad_bounds_are_reported_and_stay_inside(bounds):
    skip_without_gpu()
    torch = torch_mod()
    Q, K, V, _, _ = make(4, [100], [100], 4, 2, 64, torch.float16)
    O = torch.zeros(164, 4, 64, device="cuda").half()
    w4.w4_prompt_attention(Q, K, V, torch.tensor(bounds, device="cuda").int(), O=O[32:132])
    with pytest.raises(w4.W4Error) as e:
        w4.w4_check_device_error()
    assert e.value.status == w4.W4_ERR_DEVICE_ARG
    assert (O[:32] == 0).all() and (O[132:] == 0).all()
    w4.w4_check_device_error()   # reported once


def test_empty_calls():
    skip_without_gpu()
    torch = torch_mod()
    Q = torch.randn(0, 4, 64, device="cuda").half()
    K = torch.randn(3, 2, 64, device="cuda").half()
    assert w4.w4_prompt_attention(Q, K, K).shape == (0, 4, 64)
    Q = torch.randn(3, 4, 64, device="cuda").half()
    O, lse = w4.w4_prompt_attention(Q, K[:0], K[:0], return_lse=True)
    assert (O == 0).all() and torch.isneginf(lse).all()
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    w4.w4_prompt_attention(Q, Q[:, :2], Q[:, :2], cu)    # a batch of no sequences
    w4.w4_check_device_error()


def test_workspace_is_checked():
    skip_without_gpu()
    torch = torch_mod()
    w = way("ranges")
    with pytest.raises(w4.W4Error):
        call(w, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    q, k, Q, K, V, _, _ = w
    need = w4.w4_prompt_attention_workspace_bytes(len(q), Q.shape[1], K.shape[1], 128, Q.shape[0], K.shape[0])
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")   # of any content
    assert torch.equal(call(w, workspace=ws), call(w))
