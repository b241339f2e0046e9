"""Memory that a call allocates for its results belongs to the stream that writes it."""
import contextlib
import inspect

import numpy as np
import pytest
import torch

import eagle_tree_speculative_gb300 as E
import workloads as W

D = 128


# ---------------------------------------------------------------- on the host
def test_every_call_with_a_stream_allocates_for_it():
    calls = [f for n, f in vars(E).items() if inspect.isfunction(f) and "stream" in inspect.signature(f).parameters
             and not n.startswith("_")]
    assert len(calls) >= 15
    for f in calls:
        source = inspect.getsource(f)
        assert "torch.empty" not in source and "torch.zeros" not in source, f.__name__


def test_memory_comes_from_the_stream_and_is_marked_as_used_by_the_current_one(monkeypatch):
    events = []

    class Memory:
        def record_stream(self, s):
            events.append(("used by", s))

    @contextlib.contextmanager
    def on(s):
        events.append(("on", s))
        yield
        events.append(("off", s))

    def empty(shape, dtype, device):
        events.append("allocated")
        return Memory()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: "current")
    monkeypatch.setattr(torch, "empty", empty)
    E._empty(3, torch.int32, "cuda:0", "side")
    assert events == [("on", "side"), "allocated", ("off", "side"), ("used by", "current")]
    events.clear()
    E._empty(3, torch.int32, "cuda:0", None)
    assert events == ["allocated"]


# ---------------------------------------------------------------- on the GPU
def _bf16(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def _ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _calls():
    """name -> call(stream) of the attention calls, with inputs that are ready; results of one megabyte."""
    T, B, n, Hq, Hkv = 512, 16, 16, 16, 4
    q, k, v, cu = _bf16(T, 8, D, seed=1), _bf16(T, 2, D, seed=2), _bf16(T, 2, D, seed=3), _ints([0, 300, T])
    tq, kt, vt = _bf16(B, n, Hq, D, seed=4), _bf16(B, n, Hkv, D, seed=5), _bf16(B, n, Hkv, D, seed=6)
    kc, vc = _bf16(B, Hkv, 128, D, seed=7), _bf16(B, Hkv, 128, D, seed=8)
    parent, kv_len = _ints(np.stack([W.random_tree(n, 6, 1, b) for b in range(B)])), _ints([100] * B)
    k8, v8, ks, vs = (t[0] for t in E.kv8_cache(1, B, Hkv, 128))
    rows = _bf16(B * 100, Hkv, D, seed=9)
    E.eagle_kv8_append(rows, rows, _ints(np.arange(B + 1) * 100), _ints([0] * B), k8, v8, ks, vs)
    return {"prompt": lambda s: E.eagle_prompt_attn(q, k, v, cu, stream=s),
            "tree": lambda s: E.eagle_tree_attn(tq, kc, vc, kv_len, parent, stream=s),
            "tree_kv8": lambda s: E.eagle_tree_attn_kv8(tq, k8, v8, ks, vs, kt, vt, kv_len, parent, stream=s)}


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["prompt", "tree", "tree_kv8"])
def test_a_result_on_a_side_stream_leaves_memory_in_use_alone(name):
    call = _calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    side, now = torch.cuda.Stream(), torch.cuda.current_stream()
    # memory that the current stream is still to read, given back to the allocator
    x = torch.full_like(want, 3.0)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    y = torch.empty_like(x)
    y.copy_(x)
    del x
    out = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert (y == 3.0).all() and torch.equal(out, want)
    # a result that the current stream is still to read, given back
    now.wait_stream(side)
    torch.cuda._sleep(100_000_000)
    y.copy_(out)
    del out
    with torch.cuda.stream(side):
        other = [torch.zeros_like(want) for _ in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(y, want) and len(other) == 2


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["prompt", "tree", "tree_kv8"])
def test_a_captured_call_on_a_forked_stream(name):
    call = _calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = call(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
