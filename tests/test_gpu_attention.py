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
