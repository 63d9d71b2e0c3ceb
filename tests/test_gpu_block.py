"""A transformer block (without its norms) through the library: qkv with bias, rotary positions
in place, attention, o with residual, SwiGLU, down with residual; as a prompt, as a packed
batch, and as the next tokens of it.  Every step is checked against fp64 on the step's own
inputs, with the bounds of the steps' own tests; the block as a whole must be the same in a
captured graph."""
import pytest

import bit_weight_only_w4_b200 as w4
import profile_case
from tests import test_gpu_attention as attn
from tests import test_gpu_epilogue as epi
from tests import test_gpu_rope as rope
from tests.gpu_util import skip_without_gpu, torch_mod

pytestmark = pytest.mark.gpu

W, H, HK, D, F = 256, 4, 2, 64, 384


def layers(dtype):
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = epi.Layer(1, (H + 2 * HK) * D, W, 128, dtype=dtype)
    o, down = epi.Layer(2, W, H * D, 64, dtype=dtype), epi.Layer(3, W, F, 128, dtype=dtype)
    gate_up = epi.Layer(4, 2 * F, W, 32, True, dtype=dtype)
    bias = torch.randn((H + 2 * HK) * D, generator=g, device="cuda").to(qkv.dt)
    return qkv, o, gate_up, down, bias


def product(L, x, **kw):
    y = w4.w4a16_gemm_epi(x, L.qw, L.sc, L.zr, L.group, **kw)
    epi.check(y, epi.reference(L, x, kw.get("bias"), kw.get("activation"), kw.get("gated", False), kw.get("residual")))
    return y


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("lens", [[90], [1], [33, 1, 70, 8], [300, 17]])
def test_prompts_then_next_tokens(lens, dtype):
    skip_without_gpu()
    torch = torch_mod()
    qkv, o, gate_up, down, bias = layers(dtype)
    inv, _ = w4.w4_rope_freqs(D, 10000.0, "linear", factor=2.0)
    x = torch.randn(sum(lens), W, device="cuda").to(qkv.dt)
    cu = lambda n: torch.tensor([0] + n, device="cuda").cumsum(0).int()  # noqa: E731
    keys, values, past = None, None, [0] * len(lens)
    for now in (lens, [1] * len(lens)):    # the prompts, then one more token of each sequence
        pos = torch.cat([torch.arange(p, p + n, device="cuda") for p, n in zip(past, now)]).int()
        h = product(qkv, x, bias=bias).view(sum(now), H + 2 * HK, D)
        before = h.clone()
        qk = h[:, :H + HK]
        w4.w4_rope(qk, pos, inv, Y=qk)
        rope.check(qk, before[:, :H + HK], pos, inv, False, 1.0)
        assert torch.equal(h[:, H + HK:], before[:, H + HK:])
        k, v = h[:, H:H + HK], h[:, H + HK:]
        if keys is None:
            keys, values, cu_k = k, v, None
        else:
            join = lambda old, new: torch.cat([t for p in zip(old.split(past), new.split(now)) for t in p])  # noqa: E731
            keys, values = join(keys, k), join(values, v)
            cu_k = cu([p + n for p, n in zip(past, now)])
        past = [p + n for p, n in zip(past, now)]
        a, lse = w4.w4_prompt_attention(h[:, :H], keys, values, cu(now), cu_k, return_lse=True)
        attn.check(a, lse, attn.plain(h[:, :H], keys, values, now, past, True, D ** -0.5), qkv.dt, max(past))
        x = product(o, a.view(-1, H * D), residual=x)
        x = product(down, product(gate_up, x, activation="silu", gated=True), residual=x)
        x = x[torch.tensor([sum(now[:b + 1]) - 1 for b in range(len(now))], device="cuda")].contiguous()
    w4.w4_check_device_error()


@pytest.mark.parametrize("tokens,keys", [(200, 0), (3, 700)])
def test_block_in_a_graph(tokens, keys):
    skip_without_gpu()
    torch = torch_mod()
    block, x = profile_case.block_case(w4, torch, tokens, keys, width=256, heads=8, kv_heads=2, dim=64, inner=512)
    want = block(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(x)
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    w4.w4_check_device_error()
