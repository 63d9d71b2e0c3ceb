"""Calls on a stream that is passed allocate from that stream's pool (host logic: the library is
a stand-in that only returns W4_OK, the tensors lie in host memory, and a stand-in for
torch.cuda.stream notes which allocations happen inside it)."""
import contextlib

import pytest

import bit_weight_only_w4_b200 as w4


class Library:
    def __getattr__(self, name):
        def f(*args):
            return 1 << 12 if name.endswith(("_bytes", "_bytes_perm")) else w4.W4_OK
        f.__name__ = name
        return f


@pytest.fixture
def allocations(monkeypatch):
    """(streams under which tensors were allocated, streams that use them too, a stream, watch)."""
    import torch
    from torch.utils._python_dispatch import TorchDispatchMode
    inside, seen, used = [None], [], []

    class Stream:
        cuda_stream = 4096

    @contextlib.contextmanager
    def under(stream):
        inside.append(stream)
        yield
        inside.pop()

    class Watch(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            if "empty" in func.__name__ or "zeros" in func.__name__:
                seen.append(inside[-1])
            return func(*args, **(kwargs or {}))

    cpu = torch.device("cpu", 0)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: used.append(s))
    monkeypatch.setattr(w4, "lib", Library)
    monkeypatch.setattr(w4, "_need_cuda", lambda *t: cpu)
    monkeypatch.setattr(w4, "_cuda_index", lambda *t: 0)
    monkeypatch.setattr(w4, "_DeviceGuard", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(w4, "_on_device", lambda index, fn, *a: fn(*a))
    monkeypatch.setattr(w4, "_capture_id", lambda *a: 0)
    monkeypatch.setattr(w4, "_ws_cache", {})
    monkeypatch.setattr(w4, "_sizes", {})
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    return seen, used, Stream(), Watch


def calls():
    import torch
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    N, K, g = 32, 64, 32
    W, X, qw, sc, perm, pos = h(N, K), h(2, K), i(N * K // 8), h(K // g, N), i(K), i(5)
    bs, one, inv = torch.zeros(K // 16, N, dtype=torch.uint8), torch.zeros(1), torch.zeros(32, dtype=torch.float64)
    Q = h(5, 2, 64)
    return {
        "w4_actorder_perm": lambda s: w4.w4_actorder_perm(perm, g, stream=s),
        "w4_awq_search": lambda s: w4.w4_awq_search(W, X, g, stream=s),
        "w4_quantize_pack": lambda s: w4.w4_quantize_pack(W, None, g, stream=s),
        "w4a16_gemm": lambda s: w4.w4a16_gemm(X, qw, sc, sc, g, stream=s),
        "w4a16_gemm_perm": lambda s: w4.w4a16_gemm(X, qw, sc, sc, g, perm=perm, stream=s),
        "w4a16_gemm_noalloc": lambda s: w4.w4a16_gemm_noalloc(X, qw, sc, sc, g, stream=s),
        "w4_fp4_quantize_pack": lambda s: w4.w4_fp4_quantize_pack(W, stream=s),
        "w4a16_fp4_gemm": lambda s: w4.w4a16_fp4_gemm(X, qw, bs, one, stream=s),
        "w4_unpack_canonical": lambda s: w4.w4_unpack_canonical(qw, N, K, stream=s),
        "w4a16_gemm_epi": lambda s: w4.w4a16_gemm_epi(X, qw, sc, sc, g, gated=True, stream=s),
        "w4_rope": lambda s: w4.w4_rope(Q, pos, inv, stream=s),
        "w4_prompt_attention": lambda s: w4.w4_prompt_attention(Q, Q, Q, return_lse=True, stream=s),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_allocations_of_a_call_on_a_stream(allocations, name):
    seen, used, stream, Watch = allocations
    call = calls()[name]
    with Watch():
        call(stream)
    assert seen and all(s is stream for s in seen), seen
    assert used and set(used) == {"current"}   # outputs are kept until the current stream is done with them
