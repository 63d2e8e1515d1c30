"""Calls with an explicit stream: what the binding allocates for them belongs
to that stream, so that the caching allocator neither hands out a block that
the stream still uses nor gives it one whose fill it does not wait for. On the
CPU the library is a stub and the allocations are watched; on a GPU the calls
run late on a side stream while the current one takes and fills memory."""
import contextlib
import types

import numpy as np
import pytest
import torch
from torch.overrides import TorchFunctionMode

from ddtree_speculative_decode_b200 import lib

DEV = "cuda:0"
gpu = pytest.mark.gpu


class OnGpu(torch.Tensor):
    """A CPU tensor that passes for one on a GPU."""

    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


I32, I64, BF = torch.int32, torch.int64, torch.bfloat16


def ints(shape, dtype=I32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


def evict():
    a = (t(64, 8), t(64), ints(2, I64), ints(2), ints(2), 1, 1, 16)
    return lambda **kw: lib.cache_evict(*a, **kw)


def evict_into():
    a = (t(64, 8), t(64), ints(2, I64), ints(2), ints(2), 1, 1, 16)
    dst = {"kv": t(32, 8), "score": t(32), "off": ints(2, I64)}
    return lambda **kw: lib.cache_evict(*a, dst=dst, **kw)


def weights():
    a = (t(2, 3, 4, 64, dtype=BF), t(2, 3, 4), t(64, 64, dtype=BF), t(64), ints(2, I64), ints(2), ints(2), 0.1, 16)
    return lambda **kw: lib.cache_weights(*a, **kw)


def logprobs():
    a = (t(2, 3, 50), ints((2, 3)))
    return lambda **kw: lib.token_logprobs(*a, K=4, **kw)


def topk():
    a = (t(2, 3, 50), 4)
    return lambda **kw: lib.drafter_topk(*a, **kw)


def tree():
    a = (t(2, 3, 4), ints((2, 3, 4)), ints(2), ints(2), 8)
    return lambda **kw: lib.build_tree(*a, **kw)


def attention():
    a = (t(2, 8, 4, 80), t(64, 80), ints(2, I64), ints(2), ints((2, 8, 1)), ints(2), 64, 16, 0.1, 16)
    return lambda **kw: lib.verify_attn(*a, **kw)


def accept():
    a = (t(2, 8, 50), ints((2, 8)), ints((2, 8)), ints(2), t(64, 80), ints(2, I64), ints(2), ints(2))
    return lambda **kw: lib.accept_compact(*a, **kw)


def accept_noalloc():
    a = (t(2, 8, 50), ints((2, 8)), ints((2, 8)), ints(2), t(64, 80), ints(2, I64), ints(2), ints(2))
    return lambda **kw: lib.accept_compact_noalloc(*a, **kw)


def accept_lmhead():
    a = (t(2, 8, 64, dtype=BF), t(50, 64, dtype=BF), ints((2, 8)), ints((2, 8)), ints(2), t(64, 80), ints(2, I64), ints(2),
         ints(2))
    return lambda **kw: lib.accept_compact_lmhead(*a, **kw)


CALLS = [evict, evict_into, weights, logprobs, topk, tree, attention, accept, accept_noalloc, accept_lmhead]


@pytest.mark.parametrize("make", CALLS, ids=lambda c: c.__name__)
def test_allocations_belong_to_the_stream(make, monkeypatch):
    call = make()
    active, seen = [None], []

    @contextlib.contextmanager
    def on(stream):
        before, active[0] = active[0], stream
        yield
        active[0] = before

    class Watch(TorchFunctionMode):
        def __torch_function__(self, func, types, args=(), kwargs=None):
            if func in (torch.empty, torch.zeros, torch.empty_like, torch.zeros_like, torch.full):
                seen.append(active[0])
            return func(*args, **(kwargs or {}))

    class Stub:
        def __getattr__(self, name):
            return (lambda *a: 512) if name.endswith("_size") else (lambda *a: lib.DDT_OK)

    monkeypatch.setattr(lib, "load", lambda: Stub())
    monkeypatch.setattr(lib, "_check", lambda *a, **k: None)
    monkeypatch.setattr(lib, "_device", lambda *a, **k: contextlib.nullcontext())
    monkeypatch.setattr(lib, "_ready", lambda *a: False)
    monkeypatch.setattr(torch.cuda, "stream", on)
    side = types.SimpleNamespace(cuda_stream=7, device=torch.device("cpu"))
    with Watch():
        call(stream=side)
    assert seen and all(s is side for s in seen)


def late(side):
    """Keeps a stream busy for some milliseconds."""
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)


def take_and_fill(sizes, value, times=40):
    """Takes blocks of these sizes from the current stream's memory and fills them, again and again."""
    for _ in range(times):
        for n in sizes:
            torch.full((n,), value, dtype=torch.uint8, device=DEV)


@gpu
def test_evict_on_a_side_stream():
    layers, L, keep = 16, 6000, 2500
    g = torch.Generator(device=DEV).manual_seed(1)
    kv, score = torch.randn(layers * L, 80, device=DEV, generator=g), torch.rand(layers * L, device=DEV, generator=g)
    off = torch.zeros(1, dtype=I64, device=DEV)
    n, k = torch.tensor([L], dtype=I32, device=DEV), torch.tensor([keep], dtype=I32, device=DEV)
    size = lib.cache_evict_workspace_size(1, layers, L)
    side = torch.cuda.Stream()
    for dst in (None, {"kv": torch.zeros(layers * keep, 80, device=DEV), "score": torch.zeros(layers * keep, device=DEV),
                       "off": off, "layer_stride_rows": keep}):
        x, s, c = kv.clone(), score.clone(), n.clone()
        late(side)
        out = lib.cache_evict(x, s, off, c, k, 4, 100, L, n_layers=layers, layer_stride_rows=L, dst=dst, stream=side)
        take_and_fill([size, layers * L * 4], 0x7f)
        torch.cuda.synchronize()
        assert out["new_len"].tolist() == [keep]
        order = score.view(layers, L).clone()
        order[:, :4] = np.inf
        order[:, L - 100:] = np.inf
        want = order.sort(dim=-1, descending=True, stable=True).indices[:, :keep].sort(-1).values
        assert torch.equal(out["src"][:, 0, :keep].long(), want)
        rows, step = (x, L) if dst is None else (dst["kv"], keep)
        for la in range(layers):
            assert torch.equal(rows[la * step:la * step + keep], kv[la * L + want[la]])


@gpu
@pytest.mark.parametrize("busy", ["side", "current"])
def test_weights_on_a_side_stream(busy):
    """A workspace whose zeros come late, or are overwritten early, holds a status or counts that are none."""
    L, H, d = 3000, 64, 576
    g = torch.Generator(device=DEV).manual_seed(2)
    q, kv = torch.randn(1, 24, H, d, device=DEV, generator=g).bfloat16(), torch.randn(L, d, device=DEV, generator=g).bfloat16()
    lse = torch.full((1, 24, H), 60.0, device=DEV)
    off = torch.zeros(1, dtype=I64, device=DEV)
    cl, n = torch.tensor([L], dtype=I32, device=DEV), torch.tensor([24], dtype=I32, device=DEV)
    want, score = torch.zeros(L, device=DEV), torch.zeros(L, device=DEV)
    lib.cache_weights(q, lse, kv, want, off, cl, n, 0.04, L)
    size = lib.cache_weights_workspace_size(1, 24, H, d, L, BF)
    side = torch.cuda.Stream()
    status = torch.full((1,), 9, dtype=I32, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    take_and_fill([size], 0x7f, 1)  # what a block of that size holds
    late(side) if busy == "side" else torch.cuda._sleep(20_000_000)
    lib.cache_weights(q, lse, kv, score, off, cl, n, 0.04, L, status=status, stream=side)
    take_and_fill([size], 0x7f)
    torch.cuda.synchronize()
    assert status.tolist() == [lib.DDT_OK] and torch.equal(score, want)


@gpu
@pytest.mark.parametrize("busy", ["side", "current"])
def test_a_step_on_a_side_stream(busy):
    """Top-k, attention, accept and token log-probs on a stream of their own, without workspaces or outputs."""
    g = torch.Generator(device=DEV).manual_seed(4)
    B, N, H, V, L = 2, 24, 64, 3001, 500
    draft = torch.randn(B, 6, V, device=DEV, generator=g)
    root, cl = torch.tensor([1, 2], dtype=I32, device=DEV), torch.tensor([L, L - 100], dtype=I32, device=DEV)
    off, cap = torch.tensor([0, 700], dtype=I64, device=DEV), torch.tensor([700, 700], dtype=I32, device=DEV)
    q, kv = (torch.randn(*s, device=DEV, generator=g).bfloat16() for s in ((B, N, H, 576), (1400, 576)))
    logits = torch.randn(B, N, V, device=DEV, generator=g)
    hidden, head = (torch.randn(*s, device=DEV, generator=g).bfloat16() for s in ((B, N, 512), (V, 512)))

    def step(stream):
        def between():
            if stream is not None:
                late(stream) if busy == "side" else torch.cuda._sleep(20_000_000)

        def take():
            if stream is not None:
                take_and_fill([256, lib.verify_attn_workspace_size(B, N, H, 512, 64, 4 * L, BF),
                               lib.accept_compact_workspace_size(B, N, V)], 0x7f)

        pools, lens, outs = [kv.clone(), kv.clone()], [cl.clone(), cl.clone()], []
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        between()
        top = lib.drafter_topk(draft, 4, stream=stream)
        take()
        between()
        tr = lib.build_tree(top["logp"], top["tok"], root, cl, N, stream=stream)
        take()
        between()
        o = lib.verify_attn(q, kv, off, cl, tr["mask"], tr["n_nodes"], 512, 64, 0.04, 4 * L, stream=stream)
        take()
        between()
        a = lib.accept_compact(logits, tr["node_tok"], tr["parent"], tr["n_nodes"], pools[0], off, lens[0], cap, stream=stream)
        take()
        between()
        h = lib.accept_compact_lmhead(hidden, head, tr["node_tok"], tr["parent"], tr["n_nodes"], pools[1], off, lens[1], cap,
                                      stream=stream)
        take()
        between()
        lp = lib.token_logprobs(logits, a["out_tok"], nodes=a["acc_nodes"], K=3, stream=stream)
        take()
        torch.cuda.synchronize()
        for d in (top, tr, a, h, lp, dict(enumerate(pools + lens))):
            outs += [v.clone() for v in d.values()]
        return o, outs

    (o0, l0), want = step(None)
    (o1, l1), got = step(torch.cuda.Stream())
    assert len(want) == len(got) and [i for i, (a, b) in enumerate(zip(want, got)) if not torch.equal(a, b)] == []
    # the attention joins its parts in the order in which they end: float32 sums of at most 32 parts of values below 6
    # in another order (2 x 32 x 2^-24 x 6 = 2.3e-5), each rounded to bf16 (half a step, 2^-8, on both sides)
    assert bool(((o0.float() - o1.float()).abs() <= 2.0 ** -7 * o0.float().abs() + 2.3e-5).all())
    assert bool(((l0 - l1).abs() <= 2.3e-5).all())
