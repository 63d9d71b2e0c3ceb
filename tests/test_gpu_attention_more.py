"""More of prompt attention, with the plain form and the bound of test_gpu_attention.py: scores of
hundreds whose error stays small in every way of working, non-finite values strewn over V,
prompts packed with next tokens, and the same bits every time."""
import math

import pytest

import bit_weight_only_w4_b200 as w4
from tests.gpu_util import skip_without_gpu, torch_mod
from tests.test_gpu_attention import WAYS, call, check, make, plain, way

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("shape", ["rising", "falling", "zigzag"])
@pytest.mark.parametrize("name", WAYS)
def test_scores_of_hundreds(name, shape, dtype):
    """Every query has a common part w (signs) and keys have a multiple of it that changes along
    the sequence, so scores run over 240: rising, falling, or both by turns within a key block.
    A score's error bound d is then D 2^-23 of about 300, so the check means something: weights
    are held to 2 d < 0.01."""
    skip_without_gpu()
    torch = torch_mod()
    D, scale = 64, 0.125
    q, k, H, Hk = WAYS[name]
    same = k is None
    k = q if same else k
    dt = getattr(torch, dtype)
    Q, K, V, cu_q, cu_k = make(21, q, k, H, Hk, D, dt)
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.sign(torch.randn(D, generator=g, device="cuda"))
    at = torch.cat([torch.linspace(0, 1, n, device="cuda") if n > 1 else torch.ones(n, device="cuda") for n in k])
    step = {"rising": at, "falling": 1 - at, "zigzag": torch.frac(at * 7.3) * at}[shape] * 30
    Q = (Q.float() + w).to(dt)
    K = (0.3 * K.float() + step[:, None, None] * w).to(dt)
    ref = plain(Q, K, V, q, k, True, scale)
    assert float(ref[1].max()) > 150 and 2 * float(ref[3].max()) < 0.01
    O, lse = w4.w4_prompt_attention(Q, K, V, cu_q, None if same else cu_k, scale=scale, return_lse=True)
    check(O, lse, ref, dt, max(k))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("name", WAYS)
def test_non_finite_values_strewn_over_v(name, dtype):
    """A row's output is non-finite exactly in the columns where a key that it sees is, with the
    sign that adding them gives; everywhere else it has the bits it has without them."""
    skip_without_gpu()
    torch = torch_mod()
    w = way(name, dtype=dtype)
    q, k, Q, K, V, cu_q, cu_k = w
    clean, lse0 = call(w, return_lse=True)
    G, Tq = Q.shape[1] // K.shape[1], Q.shape[0]
    g = torch.Generator(device="cuda").manual_seed(8)
    V2 = V.clone()
    keys = torch.randperm(V.shape[0], generator=g, device="cuda")[:max(3, V.shape[0] // 60)]
    for n, (key, value) in enumerate(zip(keys.tolist(), [math.inf, -math.inf, math.nan] * V.shape[0])):
        V2[key, n % V.shape[1], (37 * n) % V.shape[2]] = value
    # what a row sees: running sums of the marks along each sequence
    marks = torch.stack([V2.isnan(), torch.isposinf(V2), torch.isneginf(V2)]).double()
    want = clean.float().clone()
    for b in range(len(q)):
        a0, b0 = int(cu_q[b]), int(cu_k[b])
        run = marks[:, b0:b0 + k[b]].cumsum(1)
        last = torch.arange(q[b], device="cuda") + k[b] - q[b]
        nan, pos, neg = (r.repeat_interleave(G, 1) > 0 for r in run[:, last])
        rows = want[a0:a0 + q[b]]
        rows[pos] = math.inf
        rows[neg] = -math.inf
        rows[nan | (pos & neg)] = math.nan
    for _ in range(4):
        O, lse = w4.w4_prompt_attention(Q, K, V2, cu_q, None if q is k else cu_k, return_lse=True)
        assert torch.equal(torch.nan_to_num(O.float(), 1e30, 2e30, -2e30), torch.nan_to_num(want, 1e30, 2e30, -2e30))
        assert torch.equal(lse, lse0)
    assert Tq == O.shape[0] and not want.isfinite().all()
    w4.w4_check_device_error()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("q_lens,k_lens", [([300, 1, 1, 1], [300, 2500, 700, 4000]), ([1, 1, 700, 1, 40], [1300, 64, 700, 5000, 3000]),
                                           ([1] * 20 + [600], [128 * i + 1 for i in range(20)] + [600])])
def test_prompts_packed_with_next_tokens(q_lens, k_lens, dtype):
    skip_without_gpu()
    torch = torch_mod()
    dt = getattr(torch, dtype)
    Q, K, V, cu_q, cu_k = make(31, q_lens, k_lens, 16, 2, 128, dt)
    O, lse = w4.w4_prompt_attention(Q, K, V, cu_q, cu_k, return_lse=True)
    w4.w4_check_device_error()
    check(O, lse, plain(Q, K, V, q_lens, k_lens, True, 128 ** -0.5), dt, max(k_lens))


@pytest.mark.parametrize("name", WAYS)
def test_the_same_bits_every_time(name):
    """No sum's order depends on which CTA or warp comes first."""
    skip_without_gpu()
    torch = torch_mod()
    w, other = way(name), way(name, seed=6)
    want = call(w, return_lse=True)
    for _ in range(10):
        call(other)
        assert all(torch.equal(a, b) for a, b in zip(call(w, return_lse=True), want))
