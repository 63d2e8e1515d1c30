"""ddt_cache_weights against the definition in 64 bits: accumulated attention
weight per cached row for whole trees, node lists, single tokens and causal
entries, on both kernels (float32 / bf16, any head count and row size), ragged
and empty caches, rows without visible keys, garbage where nothing may be
read, accumulation, statuses, graphs and streams."""
import ctypes

import numpy as np
import pytest
import torch

from ddtree_speculative_decode_b200 import build, lib

DEV = "cuda:0"
gpu = pytest.mark.gpu


def reference(c):
    """(score, error bound) in float64, NaN where nothing is written.

    A weight e^(s - lse) is off by at most a factor e^delta, with delta the
    dot product's error (a sum of d float32 terms in any order, or 16-product
    tensor-core steps of twice the unit: at most (d + 16) 2^-24 scale |q|.|k|)
    plus the exponent's: scale and log2 e are rounded, the product and the
    difference are (4 roundings of values up to |s| + |lse|, 2^-24 each), and
    2^-21 for the exponential itself. The sum of n weights in chains and
    trees adds at most (n / 16 + 48) 2^-24, decay and prev two roundings."""
    q, kv = c["q"].double(), c["kv"].double()
    B, N, H, d = q.shape
    out = torch.full((kv.shape[0],), np.nan, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b in range(B):
        n, L, o = c["n"][b], c["len"][b], c["off"][b]
        if c["nodes"] is None:
            rows = list(range(n))
        else:
            rows = []
            for i in c["nodes"][b].tolist():
                if i < 0:
                    break
                rows.append(i)
        w = torch.zeros(L, dtype=torch.float64)
        e = torch.zeros(L, dtype=torch.float64)
        keys = kv[o:o + L]
        for k, i in enumerate(rows):
            lse = c["lse"][b, i].double()[:, None]
            s = c["scale"] * (q[b, i] @ keys.T)
            mag = c["scale"] * (q[b, i].abs() @ keys.abs().T)
            p = torch.exp(s - lse)
            p[(lse == -np.inf).expand_as(p)] = 0
            if c["causal"]:
                p[:, max(0, L - len(rows) + 1 + k):] = 0
            delta = (d + 16) * 2.0 ** -24 * mag + 4 * 2.0 ** -24 * (s.abs() + lse.abs()) + 2.0 ** -21
            delta = torch.where(p > 0, delta, torch.zeros_like(p))
            w += p.sum(0)
            e += (p * torch.expm1(delta)).sum(0)
        e += w * (len(rows) * H / 16 + 48) * 2.0 ** -24
        if c["prev"] is not None:
            pv = c["prev"][o:o + L].double()
            w = w + c["decay"] * pv
            e = e + 2 * 2.0 ** -24 * (w.abs() + c["decay"] * pv.abs())
        out[o:o + L] = w
        tol[o:o + L] = e + 1e-37  # results below float32's normal range may flush to zero
    return out, tol


def make(lens, N, H, d, dtype, seed, nodes=None, causal=False, n=None, prev=True, decay=0.9, kv_scale=1.0, scale=None):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    off, at = [], 3
    for L in lens:
        off.append(at)
        at += L + 4
    q = torch.randn(B, N, H, d, generator=g).to(dtype)
    kv = torch.randn(at, d, generator=g).mul(kv_scale).to(dtype)
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    lse = torch.zeros(B, N, H)
    for b, L in enumerate(lens):
        if L:
            lse[b] = torch.logsumexp(scale * (q[b].float() @ kv[off[b]:off[b] + L].float().T), -1)
    return {"q": q, "kv": kv, "lse": lse, "off": off, "len": list(lens), "n": [N] * B if n is None else list(n),
            "nodes": nodes, "causal": causal, "scale": scale, "decay": decay,
            "prev": torch.rand(at, generator=g) if prev else None}


def run(c, max_len=None, workspace=None, status=None, **kw):
    """The call's scores (a fill of -7 where nothing was written)."""
    i32 = dict(dtype=torch.int32, device=DEV)
    score = torch.full((c["kv"].shape[0],), -7.0, device=DEV)
    nodes = None if c["nodes"] is None else c["nodes"].to(DEV, torch.int32)
    prev = None if c["prev"] is None else c["prev"].to(DEV)
    lib.cache_weights(c["q"].to(DEV), c["lse"].to(DEV), c["kv"].to(DEV), score, torch.tensor(c["off"], device=DEV),
                      torch.tensor(c["len"], **i32), torch.tensor(c["n"], **i32), c["scale"],
                      max(c["len"]) if max_len is None else max_len, nodes=nodes, causal=c["causal"], prev=prev,
                      decay=c["decay"], workspace=workspace, status=status, **kw)
    torch.cuda.synchronize()
    return score.cpu()


def check(c, **kw):
    B = len(c["len"])
    status = torch.full((B,), 9, dtype=torch.int32, device=DEV)
    got = run(c, status=status, **kw)
    ref, tol = reference(c)
    assert status.tolist() == [lib.DDT_OK] * B
    wrote = ~torch.isnan(ref)
    assert bool((got[~wrote] == -7.0).all()), "a row outside the caches was written"
    err = (got[wrote].double() - ref[wrote]).abs()
    assert bool((err <= tol[wrote]).all()), (float((err / tol[wrote]).max()), float(err.max()))
    return got


def paths(B, N, M, seed, longest=9):
    r = np.random.default_rng(seed)
    out = torch.full((B, M), -1, dtype=torch.int32)
    for b in range(B):
        m = int(r.integers(1, min(N, M, longest) + 1))
        out[b, :m] = torch.from_numpy(np.concatenate([[0], 1 + np.sort(r.permutation(N - 1)[:m - 1])]).astype(np.int32))
    return out


@gpu
@pytest.mark.parametrize("L", [0, 1, 2, 63, 64, 65, 129, 500])
@pytest.mark.parametrize("N,H,d", [(1, 4, 80), (9, 3, 33), (5, 1, 1), (2, 2, 1024)])
def test_f32(L, N, H, d):
    check(make([L, max(0, L - 1)], N, H, d, torch.float32, L + N))


@gpu
@pytest.mark.parametrize("L", [0, 1, 127, 128, 129, 255, 256, 257, 700])
@pytest.mark.parametrize("N", [1, 2, 5])
def test_mla_rows(L, N):
    check(make([L, max(0, L - 1), L + 1], N, 64, 576, torch.bfloat16, L + N))


@gpu
@pytest.mark.parametrize("H", [1, 2, 7, 8, 16, 20, 40, 72, 100, 128, 130, 260])
def test_head_counts(H):
    check(make([300, 31], 5, H, 576, torch.bfloat16, H))
    check(make([300, 31], 5, H, 576, torch.bfloat16, H, nodes=paths(2, 5, 5, H), causal=True))


@gpu
@pytest.mark.parametrize("d", [8, 64, 128, 192, 200, 512, 576, 640])
def test_row_sizes(d):
    check(make([400, 90], 6, 16, d, torch.bfloat16, d, nodes=paths(2, 6, 6, d), causal=True))


@gpu
@pytest.mark.parametrize("dtype,d", [(torch.float32, 33), (torch.float32, 40), (torch.float32, 576), (torch.bfloat16, 20),
                                     (torch.bfloat16, 104), (torch.bfloat16, 640)])
@pytest.mark.parametrize("N,H", [(2, 16), (3, 11), (9, 16), (19, 15)])
def test_cuda_core_tiles(N, H, d, dtype):
    """One to three tiles of rows, of both sizes, over keys that end before, at and behind a tile's end."""
    check(make([127, 128, 129, 1, 300], N, H, d, dtype, N + d))
    check(make([127, 64, 65, 2, 300], N, H, d, dtype, N + d, nodes=paths(5, N, N, d), causal=True), max_len=100)


@gpu
@pytest.mark.parametrize("dtype,H,d", [(torch.float32, 4, 80), (torch.bfloat16, 64, 576), (torch.bfloat16, 16, 576)])
@pytest.mark.parametrize("causal", [False, True])
def test_node_lists(dtype, H, d, causal):
    """Paths, an empty list, a full one, a node listed twice, more entries than nodes, more entries than rows."""
    nodes = torch.tensor([[0, 2, 5, 7, -1, 3, 3, 1, 2], [-1, 0, 1, 2, 3, 4, 5, 6, 7], [7, 6, 5, 4, 3, 2, 1, 0, 0],
                          [4, 4, 4, -5, 0, 0, 0, 0, 0], [0, 1, 2, 3, 4, 5, 6, 7, 7]])
    check(make([90, 50, 260, 40, 3], 8, H, d, dtype, 3, nodes=nodes, causal=causal))


@gpu
@pytest.mark.parametrize("dtype,H,d", [(torch.float32, 4, 80), (torch.bfloat16, 64, 576)])
def test_every_node_causal(dtype, H, d):
    check(make([200, 7, 12], 10, H, d, dtype, 5, causal=True, n=[10, 10, 0]))
    check(make([200, 7, 12], 10, H, d, dtype, 5, causal=False, n=[3, 0, 9]))


@gpu
@pytest.mark.parametrize("dtype,H,d", [(torch.float32, 4, 80), (torch.bfloat16, 64, 576)])
def test_accumulation(dtype, H, d):
    check(make([150], 3, H, d, dtype, 1, prev=False))
    check(make([150], 3, H, d, dtype, 1, decay=0.0))
    check(make([150], 3, H, d, dtype, 1, decay=1.0))
    c = make([150, 80], 3, H, d, dtype, 2, decay=0.5)
    want = check(c)
    i32 = dict(dtype=torch.int32, device=DEV)
    score = c["prev"].to(DEV)  # in place
    lib.cache_weights(c["q"].to(DEV), c["lse"].to(DEV), c["kv"].to(DEV), score, torch.tensor(c["off"], device=DEV),
                      torch.tensor(c["len"], **i32), torch.tensor(c["n"], **i32), c["scale"], 150, prev=score, decay=0.5)
    wrote = want != -7.0
    assert torch.equal(score.cpu()[wrote], want[wrote])
    assert torch.equal(score.cpu()[~wrote], c["prev"][~wrote])


@gpu
@pytest.mark.parametrize("dtype,H,d", [(torch.float32, 4, 80), (torch.bfloat16, 64, 576), (torch.bfloat16, 20, 576)])
def test_garbage_where_nothing_is_read(dtype, H, d):
    """NaN and infinities in unlisted rows, between the caches, in keys no entry sees, and rows with lse -inf."""
    nodes = torch.tensor([[1, 4, -1, 0], [3, -1, -1, -1]])
    c = make([140, 70], 6, H, d, dtype, 4, nodes=nodes, causal=True)
    clean = check(c)
    for i in (0, 2, 3, 5):
        c["q"][0, i] = np.nan
        c["lse"][0, i] = np.nan
    c["q"][1, [0, 1, 2, 4, 5]] = np.inf
    for row in list(range(3)) + list(range(143, 147)) + list(range(217, c["kv"].shape[0])):
        c["kv"][row] = np.nan
    assert torch.equal(run(c), clean)
    c["lse"][0, 4, 1:] = -np.inf
    got = run(c)
    ref, tol = reference({**c, "q": torch.nan_to_num(c["q"]), "kv": torch.nan_to_num(c["kv"])})
    wrote = ~torch.isnan(ref)
    assert bool(((got[wrote].double() - ref[wrote]).abs() <= tol[wrote]).all())
    c["q"][0, 4, 1:] = np.nan  # a row without visible keys counts for nothing, whatever its query holds
    assert torch.equal(run(c), got)


@gpu
@pytest.mark.parametrize("dtype,H,d", [(torch.float32, 4, 80), (torch.bfloat16, 64, 576)])
def test_bad_keys_stay_to_themselves(dtype, H, d):
    """A NaN key makes its own score NaN and no other."""
    c = make([200], 3, H, d, dtype, 4)
    clean = run(c)
    c["kv"][c["off"][0] + 77] = np.nan
    got = run(c)
    others = torch.ones_like(got, dtype=torch.bool)
    others[c["off"][0] + 77] = False
    assert torch.equal(got[others], clean[others]) and bool(torch.isnan(got[~others]).all())


@gpu
@pytest.mark.parametrize("dtype,H,d", [(torch.float32, 4, 80), (torch.bfloat16, 64, 576)])
def test_large_logits(dtype, H, d):
    """Peaked attention: logits of +-60, weights from 1 down to nothing."""
    check(make([300], 4, H, d, dtype, 8, scale=1.5 / np.sqrt(d) * 8))


@gpu
@pytest.mark.parametrize("lens,N,H", [([4096], 64, 64), ([6000, 1, 2500, 8192], 1, 64), ([3000] * 9, 33, 64), ([20000], 40, 16),
                                      ([70], 600, 64), ([513] * 40, 2, 64)])
def test_bf16_splits(lens, N, H):
    """Shapes that split the rows and keys differently: few keys and many rows, many keys and few rows, many requests."""
    check(make(lens, N, H, 576, torch.bfloat16, N, kv_scale=0.5))


@gpu
def test_longer_than_announced():
    for dtype, H, d in ((torch.float32, 4, 80), (torch.bfloat16, 64, 576)):
        check(make([1000, 30], 3, H, d, dtype, 8), max_len=64)


@gpu
def test_many_requests():
    lens = [int(x) for x in np.random.default_rng(0).integers(0, 40, 1500)]
    check(make(lens, 1, 8, 64, torch.bfloat16, 1))


@gpu
@pytest.mark.parametrize("dtype,H,d", [(torch.float32, 4, 80), (torch.bfloat16, 64, 576)])
def test_statuses(dtype, H, d):
    nodes = torch.tensor([[0, 1, -1], [0, 4, -1], [0, -1, 9], [0, 1, 2], [0, 1, 2], [0, 1, 2]])
    c = make([50, 50, 50, 50, 50, 50], 4, H, d, dtype, 1, nodes=nodes, n=[4, 4, 4, 5, -1, 4])
    rows = c["kv"].shape[0]
    c["off"][5] = rows - 49
    status = torch.full((6,), 9, dtype=torch.int32, device=DEV)
    got = run(c, status=status)
    bad = lib.DDT_ERR_INPUT
    assert status.tolist() == [0, bad, 0, bad, bad, lib.DDT_ERR_BOUNDS]
    for b in (1, 3, 4):
        assert bool((got[c["off"][b]:c["off"][b] + 50] == -7.0).all())
    assert bool((got[rows - 49:] == -7.0).all())
    ok = {**c, "off": [c["off"][0], c["off"][2]], "len": [50, 50], "n": [4, 4], "nodes": nodes[[0, 2]], "q": c["q"][[0, 2]],
          "lse": c["lse"][[0, 2]]}
    ref, tol = reference(ok)
    wrote = ~torch.isnan(ref)
    assert bool(((got[wrote].double() - ref[wrote]).abs() <= tol[wrote]).all())


@gpu
@pytest.mark.parametrize("dtype,H,d", [(torch.float32, 4, 80), (torch.bfloat16, 64, 576)])
def test_offsets_at_the_64_bit_limit_are_out_of_bounds(dtype, H, d):
    c = make([50, 50], 2, H, d, dtype, 1)
    c["off"][0] = 2 ** 63 - 1
    status = torch.full((2,), 9, dtype=torch.int32, device=DEV)
    got = run(c, status=status)
    assert status.tolist() == [lib.DDT_ERR_BOUNDS, 0]
    wrote = got != -7.0
    assert int(wrote.sum()) == 50 and bool(wrote[c["off"][1]:c["off"][1] + 50].all())


@gpu
def test_repeats_streams_and_graphs():
    """The same bits on every run, with a workspace that is used again and again, on another stream, from two graphs."""
    c = make([2000, 900, 1], 24, 64, 576, torch.bfloat16, 5, nodes=paths(3, 24, 24, 5), causal=True)
    n = lib.cache_weights_workspace_size(3, 24, 64, 576, 2000, torch.bfloat16)
    ws = torch.zeros(max(n, 256), dtype=torch.uint8, device=DEV)
    first = check(c, workspace=ws)
    for _ in range(3):
        assert torch.equal(run(c, workspace=ws), first)
    assert torch.equal(run(c), first)
    i32 = dict(dtype=torch.int32, device=DEV)
    t = {k: c[k].to(DEV) for k in ("q", "lse", "kv", "prev")}
    off, cl, nn = torch.tensor(c["off"], device=DEV), torch.tensor(c["len"], **i32), torch.tensor(c["n"], **i32)
    nodes = c["nodes"].to(DEV)

    def call(score, **kw):
        lib.cache_weights(t["q"], t["lse"], t["kv"], score, off, cl, nn, c["scale"], 2000, nodes=nodes, causal=True,
                          prev=t["prev"], decay=c["decay"], **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = torch.full((c["kv"].shape[0],), -7.0, device=DEV)
    torch.cuda.synchronize()
    call(s, stream=side)
    side.synchronize()
    assert torch.equal(s.cpu(), first)
    graphs = []
    for _ in range(2):  # two graphs over one workspace, replayed in turn
        s = torch.full((c["kv"].shape[0],), -7.0, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(s, workspace=ws)
        graphs.append((g, s))
    for _ in range(2):
        for g, s in graphs:
            s.fill_(-7.0)
            g.replay()
    torch.cuda.synchronize()
    for g, s in graphs:
        assert torch.equal(s.cpu(), first)


@gpu
def test_bindings_refusals():
    c = make([50], 3, 4, 80, torch.float32, 1)
    i32 = dict(dtype=torch.int32, device=DEV)
    a = [c["q"].to(DEV), c["lse"].to(DEV), c["kv"].to(DEV), torch.zeros(c["kv"].shape[0], device=DEV),
         torch.tensor(c["off"], device=DEV), torch.tensor([50], **i32), torch.tensor([3], **i32), 0.1, 50]

    def swap(i, v):
        return a[:i] + [v] + a[i + 1:]

    for i, v in ((0, a[0].cpu()), (0, a[0].transpose(1, 2)), (1, a[1][:, :2]), (2, a[2][:, :40]), (3, a[3][:-1]), (6, a[6][:0])):
        with pytest.raises(ValueError):
            lib.cache_weights(*swap(i, v))
    for i, v in ((0, a[0].half()), (2, a[2].bfloat16()), (4, a[4].int()), (5, a[5].long()), (1, a[1].double())):
        with pytest.raises(TypeError):
            lib.cache_weights(*swap(i, v))
    for v in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(lib.DDTError):
            lib.cache_weights(*swap(7, v))
    with pytest.raises(lib.DDTError):
        lib.cache_weights(*a, decay=float("nan"), prev=a[3])
    with pytest.raises(lib.DDTError):
        lib.cache_weights(*swap(8, -1))


def test_host_validation():
    build.build()
    so = lib.load()
    p = ctypes.c_void_p(256)

    def call(q=p, lse=p, kv=p, rows=100, off=p, cl=p, nodes=None, nn=p, B=2, N=3, M=0, H=4, d=80, scale=0.1, ml=50, dt=0,
             decay=1.0, score=p):
        return so.ddt_cache_weights(q, lse, kv, rows, off, cl, nodes, nn, B, N, M, H, d, scale, 0, ml, dt, None, decay, score,
                                    None, None, 0, None)

    bad, uns = lib.DDT_ERR_INVALID_ARG, lib.DDT_ERR_UNSUPPORTED
    assert call(q=None) == call(lse=None) == call(kv=None) == call(off=None) == call(cl=None) == call(nn=None) == bad
    assert call(score=None) == call(rows=0) == call(B=0) == call(N=0) == call(H=0) == call(d=0) == call(ml=-1) == bad
    assert call(dt=2) == call(nodes=p, M=0) == call(scale=0.0) == call(scale=float("nan")) == call(decay=float("inf")) == bad
    assert call(q=ctypes.c_void_p(258)) == call(kv=ctypes.c_void_p(257)) == bad
    assert call(d=1025) == call(rows=1 << 31) == call(B=1 << 20, N=1 << 12) == call(nodes=p, M=1 << 30) == uns
