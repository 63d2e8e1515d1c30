"""Rare paths of the token-score and cache-budget calls: what ordinary inputs
seldom reach, each against a plain computation."""
import ctypes

import pytest
import torch

from ddtree_speculative_decode_b200 import build, lib, spec_engine, synth
from test_gpu_logprobs import check

DEV = "cuda:0"
gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [1, 8, 32])
def test_rows_of_few_values_on_every_sm(K, dtype):
    """Rows whose best values are many and equal are read again under a count of the keys found so far, which several
    warps add to and all of them branch on: hundreds of such rows at once, every result of every run the lowest
    tokens of the largest value."""
    V, N, distinct = 20011, 600, 5
    g = torch.Generator(device=DEV).manual_seed(K)
    x = torch.randint(0, distinct, (1, N, V), device=DEV, generator=g)
    x[0, ::3] = x[0, ::3].sort(-1).values  # rising: the bound moves with the row
    tok = torch.zeros(1, N, dtype=torch.int32, device=DEV)
    # distinct sorting keys: the value, then the lower token
    want = torch.topk(x * V + (V - 1 - torch.arange(V, device=DEV)), K, dim=-1).indices.int()
    logits = x.to(dtype)
    for _ in range(10):
        out = lib.token_logprobs(logits, tok, K=K)
        assert torch.equal(out["top_tok"], want)
        assert bool((out["status"] == lib.DDT_OK).all())


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [0, 8])
def test_logits_around_a_million(K, dtype):
    """Rows whose running maximum passes +-1e6, where the sums' reference changes, between two loads of one thread:
    by less and by more than the reference's slack, for one thread and for all. Tolerances of test_gpu_logprobs."""
    V, step = 40000, 4096 if dtype == torch.float32 else 8192  # a thread's next element: `step` later
    g = torch.Generator(device=DEV).manual_seed(5)
    rows = []
    for lo, hi in ((999998.0, 1000002.0), (999999.9375, 1000000.0), (999990.0, 1000010.0), (999980.0, 1000040.0),
                   (-1000002.0, -999998.0), (-1000000.0, -999999.9375), (1000002.0, 999998.0), (5.0, 1000003.0)):
        one = torch.full((V,), lo - 30.0, device=DEV)
        one[100], one[100 + step] = lo, hi
        every = torch.full((V,), lo, device=DEV) - torch.rand(V, device=DEV, generator=g) * 4
        every[step:] += hi - lo
        rows += [one, every]
    logits = torch.stack(rows).to(dtype)[None]
    tok = torch.tensor([[100, 100 + step] * (len(rows) // 2)])
    check(logits, tok, K=K)


@gpu
@pytest.mark.parametrize("lens,N,H", [([700, 90], 1, 64), ([700, 90], 40, 64), ([300] * 3, 5, 8)])
def test_weights_workspace_that_holds_a_timeout(lens, N, H):
    """No work until the workspace is zeroed: the status of every request, no score touched, then the scores of a call
    with a fresh workspace, bit for bit. One, several and no shares of the query rows."""
    g = torch.Generator(device=DEV).manual_seed(N)
    i32 = dict(dtype=torch.int32, device=DEV)
    B, rows = len(lens), sum(lens)
    q, kv = (torch.randn(*s, device=DEV, generator=g).bfloat16() for s in ((B, N, H, 576), (rows, 576)))
    lse, prev = torch.full((B, N, H), 30.0, device=DEV), torch.rand(rows, device=DEV, generator=g)
    off = torch.tensor([sum(lens[:b]) for b in range(B)], device=DEV)
    cl, n = torch.tensor(lens, **i32), torch.tensor([N] * B, **i32)
    ws = torch.zeros(lib.cache_weights_workspace_size(B, N, H, 576, max(lens), torch.bfloat16), dtype=torch.uint8, device=DEV)

    def call(ws):
        score, status = prev.clone(), torch.full((B,), 9, **i32)
        lib.cache_weights(q, lse, kv, score, off, cl, n, 0.04, max(lens), prev=score, decay=0.5, status=status, workspace=ws)
        return score, status.tolist()

    want, status = call(None)
    assert status == [lib.DDT_OK] * B and not torch.equal(want, prev)
    ws[:4].view(torch.int32)[0] = lib.DDT_ERR_TIMEOUT
    for _ in range(2):
        score, status = call(ws)
        assert status == [lib.DDT_ERR_TIMEOUT] * B and torch.equal(score, prev)
    assert int(ws[:4].view(torch.int32)[0]) == lib.DDT_ERR_TIMEOUT and not bool(ws[4:].any())
    ws.zero_()
    score, status = call(ws)
    assert status == [lib.DDT_OK] * B and torch.equal(score, want)
    assert not bool(ws[:256].any())


@gpu
@pytest.mark.parametrize("lens,N", [([16384] * 4, 64), ([4096], 64), ([9000] * 60, 1)])
def test_weights_status_word_set_at_any_time(lens, N):
    """The status word is set from another stream before, while and after the kernel runs (waits look at it only when
    they last long). Every score is then either untouched or the right one, bit for bit, and the workspace works again
    once it is zeroed."""
    H, B, rows = 64, len(lens), sum(lens)
    g = torch.Generator(device=DEV).manual_seed(N)
    i32 = dict(dtype=torch.int32, device=DEV)
    q, kv = (torch.randn(*s, device=DEV, generator=g).bfloat16() for s in ((B, N, H, 576), (rows, 576)))
    lse, prev = torch.full((B, N, H), 30.0, device=DEV), torch.rand(rows, device=DEV, generator=g)
    off = torch.tensor([sum(lens[:b]) for b in range(B)], device=DEV)
    cl, n = torch.tensor(lens, **i32), torch.tensor([N] * B, **i32)
    ws = torch.zeros(lib.cache_weights_workspace_size(B, N, H, 576, max(lens), torch.bfloat16), dtype=torch.uint8, device=DEV)
    word = ws[:4].view(torch.int32)

    def call(score):
        lib.cache_weights(q, lse, kv, score, off, cl, n, 0.04, max(lens), prev=score, decay=0.5, workspace=ws)

    want = prev.clone()
    call(want)
    assert not bool((want == prev).any())
    # the call behind a spin of `ahead` cycles, the word behind others: before, during and after the kernel
    side, ahead = torch.cuda.Stream(), 2_000_000
    for k in range(16):
        score = prev.clone()
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(ahead)
        with torch.cuda.stream(side):
            torch.cuda._sleep(ahead + 20_000 * (k - 5))
            word.fill_(lib.DDT_ERR_TIMEOUT)
        call(score)
        torch.cuda.synchronize()
        done = score == want
        assert bool((done | (score == prev)).all())
        ws.zero_()
        again = prev.clone()
        call(again)
        assert torch.equal(again, want)


@gpu
@pytest.mark.parametrize("name,index,value", [("cache_weights", 6, -1), ("cache_evict", 4, -1)])
def test_engine_notices_a_skipped_call(name, index, value, monkeypatch):
    """A request that the device skips (here: for a negative count) raises; the engine's length stays the cache's."""
    real = getattr(lib, name)
    eng = spec_engine.TinyMLAEngine(synth.tiny_mla_weights(), 64, cache_budget=4, sink=1, recent=1)
    for t in (3, 14, 15, 92):
        eng._one_row(t)
    kv, score = eng.kv.clone(), eng.score.clone()
    monkeypatch.setattr(lib, name, lambda *a, **k: real(*a[:index], torch.full_like(a[index], value), *a[index + 1:], **k))
    with pytest.raises(RuntimeError, match="error"):
        eng._one_row(65)
    assert eng.length == 5 and eng.evicted == 0
    for la in range(eng.n_layers):
        rows = slice(la * eng.stride, la * eng.stride + 4)
        assert torch.equal(eng.kv[rows], kv[rows])
        if name == "cache_weights":
            assert torch.equal(eng.score[rows], score[rows])
    monkeypatch.setattr(lib, name, real)


@gpu
@pytest.mark.parametrize("dtype,H,d", [(torch.float32, 2, 40), (torch.bfloat16, 8, 64)])
@pytest.mark.parametrize("most", [2 ** 31 - 1, 2 ** 31 - 300])
def test_weights_with_the_loosest_bound(most, dtype, H, d):
    """max_cache_len only has to be a bound: any one gives the same scores, for many requests as well."""
    B, L = 200, 150
    g = torch.Generator(device=DEV).manual_seed(3)
    i32 = dict(dtype=torch.int32, device=DEV)
    q, kv = (torch.randn(*s, device=DEV, generator=g).to(dtype) for s in ((B, 2, H, d), (B * L, d)))
    lse = torch.full((B, 2, H), 8.0, device=DEV)
    off = torch.arange(B, device=DEV) * L
    cl, n = torch.randint(1, L + 1, (B,), generator=g, **i32), torch.full((B,), 2, **i32)
    got = []
    for m in (L, most):
        status, score = torch.full((B,), 9, **i32), torch.full((B * L,), -7.0, device=DEV)
        lib.cache_weights(q, lse, kv, score, off, cl, n, 0.1, m, status=status)
        assert status.tolist() == [lib.DDT_OK] * B
        got.append(score)
    assert torch.equal(*got)


def test_logprobs_entries_that_32_bits_cannot_count():
    """Entry numbers are counted past the last one, by up to a launch's CTAs: refused before anything is launched."""
    build.build()
    p = ctypes.c_void_p(256)
    for B, M in ((1, 2 ** 31 - 1), (2, 2 ** 30 - 100), (1, 2 ** 31 - 2 ** 16)):
        assert lib.load().ddt_token_logprobs(p, 1, 8, 8, None, p, B, M, M, 0, p, None, None, None, None,
                                             None) == lib.DDT_ERR_UNSUPPORTED


def test_weights_rows_that_32_bits_cannot_count():
    """As above, for (entry, head) rows, which the kernels take in tiles."""
    build.build()
    p = ctypes.c_void_p(256)
    for N, M, H, nodes in ((2 ** 31 - 1, 0, 1, None), (2 ** 28 - 1, 0, 8, None), (100, 2 ** 28 - 1, 8, p)):
        assert lib.load().ddt_cache_weights(p, p, p, 100, p, p, nodes, p, 1, N, M, H, 8, 0.1, 0, 50, 0, None, 1.0, p, None,
                                            None, 0, None) == lib.DDT_ERR_UNSUPPORTED


def test_evict_refuses_before_it_selects():
    """More CTAs than a launch may have for the move: refused before the selection writes statuses and lists that no
    move follows."""
    build.build()
    p, q = ctypes.c_void_p(256), ctypes.c_void_p(1 << 20)
    for kd, rows, B, mk in ((q, 100, 64, 1 << 30), (None, 0, 1 << 20, 8)):  # copied, in place; rows of 1 MB
        assert lib.load().ddt_cache_evict(p, 100, 0, 1 << 18, p, 1, 0, p, p, p, 0, 0, B, 50, kd, rows, kd, 0, kd, p, p, mk,
                                          None, p, 1 << 40, None) == lib.DDT_ERR_UNSUPPORTED
