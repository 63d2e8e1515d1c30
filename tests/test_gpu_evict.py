"""ddt_cache_evict against a plain selection on the host: which rows stay
(sink, recent window, best scores, ties to the lower row, NaN and infinite
scores), their order, the rows and scores that move, in place and into another
region, on several layers and ragged requests, and the device statuses."""
import ctypes

import numpy as np
import pytest
import torch

from ddtree_speculative_decode_b200 import build, lib

DEV = "cuda:0"
gpu = pytest.mark.gpu


def kept_rows(score, keep, sink, recent):
    """Plain selection, float64 order with NaN below everything."""
    n = len(score)
    if n <= keep:
        return np.arange(n)
    s = score.astype(np.float64) + 0.0
    rank = sorted(range(n), key=lambda i: (not (i < sink or i >= n - recent), np.isnan(s[i]),
                                           0.0 if np.isnan(s[i]) else -s[i], i))
    return np.sort(np.array(rank[:keep], dtype=np.int64))


def make(lens, layers, d, dtype, seed, gap=3):
    g = torch.Generator().manual_seed(seed)
    off, at = [], 2
    for n in lens:
        off.append(at)
        at += n + gap
    kv = torch.randn(layers * at, d, generator=g).to(dtype)
    score = torch.randn(layers * at, generator=g).mul(2).exp()
    return kv, score, off, at


def run(kv, score, lens, off, stride, keep, sink, recent, layers, dst=False, max_len=None, **kw):
    """Runs the call and checks everything it wrote or had to leave alone."""
    B, d = len(lens), kv.shape[1]
    i32 = dict(dtype=torch.int32, device=DEV)
    dkv, dscore = kv.to(DEV), score.to(DEV)
    cl = torch.tensor(lens, **i32)
    args = (dkv, dscore, torch.tensor(off, device=DEV), cl, torch.tensor(keep, **i32), sink, recent,
            max(lens) if max_len is None else max_len)
    status = torch.full((B,), 99, **i32)
    out = {"src": torch.full((layers, B, max(1, max(max(keep), 1))), 77, **i32)}
    want = [min(n, k) for n, k in zip(lens, keep)]
    d2 = None
    if dst:
        doff, at = [], 1
        for n in want:
            doff.append(at)
            at += n + 2
        d2 = {"kv": torch.full((layers * at, d), 5.0, dtype=kv.dtype, device=DEV),
              "score": torch.full((layers * at,), -3.0, device=DEV), "off": torch.tensor(doff, device=DEV),
              "layer_stride_rows": at}
    lib.cache_evict(*args, n_layers=layers, layer_stride_rows=stride, dst=d2, out=out, status=status, **kw)
    torch.cuda.synchronize()
    ref_kv, ref_score = (kv.clone(), score.clone()) if not dst else \
        (torch.full((layers * at, d), 5.0, dtype=kv.dtype), torch.full((layers * at,), -3.0))
    to_off, to_stride = (off, stride) if not dst else (doff, at)
    touched = torch.ones(ref_kv.shape[0], dtype=torch.bool)  # rows whose contents are specified
    for la in range(layers):
        for b in range(B):
            a = la * stride + off[b]
            idx = kept_rows(score[a:a + lens[b]].numpy(), keep[b], sink, recent)
            src = out["src"][la, b].cpu().numpy()
            assert np.array_equal(src[:want[b]], idx), (la, b)
            assert np.all(src[want[b]:] == -1)
            to = la * to_stride + to_off[b]
            ref_kv[to:to + want[b]] = kv[a + torch.from_numpy(idx)]
            ref_score[to:to + want[b]] = score[a + torch.from_numpy(idx)]
            if not dst:
                touched[to + want[b]:to + lens[b]] = False
    got_kv, got_score = (dkv, dscore) if not dst else (d2["kv"], d2["score"])
    as_bits = (lambda t: t.view(torch.int16)) if kv.dtype == torch.bfloat16 else (lambda t: t.view(torch.int32))
    assert torch.equal(as_bits(got_kv.cpu())[touched], as_bits(ref_kv)[touched])
    assert torch.equal(got_score.cpu().view(torch.int32)[touched], ref_score.view(torch.int32)[touched])
    if dst:
        assert torch.equal(as_bits(dkv.cpu()), as_bits(kv)) and torch.equal(dscore.cpu().view(torch.int32),
                                                                            score.view(torch.int32))
        assert cl.tolist() == list(lens)
    assert out["new_len"].tolist() == want
    assert status.tolist() == [0] * B


@gpu
@pytest.mark.parametrize("dst", [False, True])
@pytest.mark.parametrize("n,keep,sink,recent", [
    (1, 1, 0, 0), (1, 0, 0, 0), (2, 1, 0, 0), (2, 1, 1, 0), (2, 1, 0, 1), (5, 4, 0, 0), (33, 7, 2, 3), (63, 31, 0, 31),
    (64, 32, 32, 0), (100, 99, 4, 16), (1000, 500, 4, 100), (1024, 1023, 0, 0), (1025, 1, 0, 0), (4095, 2000, 1, 64),
    (4097, 4096, 3, 5), (9000, 0, 0, 0), (20000, 10001, 4, 4000)])
def test_one_request(n, keep, sink, recent, dst):
    kv, score, off, at = make([n], 1, 20, torch.float32, n + keep)
    run(kv, score, [n], off, at, [keep], sink, recent, 1, dst=dst)


@gpu
@pytest.mark.parametrize("dst", [False, True])
@pytest.mark.parametrize("d,dtype", [(576, torch.bfloat16), (80, torch.float32), (2, torch.bfloat16), (8, torch.bfloat16),
                                     (66, torch.bfloat16), (1, torch.float32), (520, torch.bfloat16)])
def test_row_sizes_and_layers(d, dtype, dst):
    lens, keep = [300, 0, 41, 777, 64, 1], [100, 10, 50, 640, 63, 0]
    kv, score, off, at = make(lens, 3, d, dtype, d)
    run(kv, score, lens, off, at, keep, 0, 0, 3, dst=dst)
    run(kv, score, lens, off, at, [max(k, 24) for k in keep], 4, 20, 3, dst=dst)


@gpu
@pytest.mark.parametrize("dst", [False, True])
def test_longer_than_the_selection_holds(dst):
    """More rows than shared memory holds keys for, and a cache longer than announced."""
    n = 60001
    kv, score, off, at = make([n], 1, 4, torch.float32, 3)
    run(kv, score, [n], off, at, [n // 2], 4, 100, 1, dst=dst)
    run(kv[:3000], score[:3000], [2500], [7], 3000, [1200], 4, 100, 1, dst=dst, max_len=100)


@gpu
@pytest.mark.parametrize("dst", [False, True])
@pytest.mark.parametrize("kind", ["equal", "few", "zeros", "nan", "inf", "negative", "rising", "falling"])
def test_scores(kind, dst):
    n = 5000
    kv, score, off, at = make([n, n], 2, 12, torch.float32, 4)
    i = torch.arange(score.numel())
    if kind == "equal":
        score[:] = 0.5
    elif kind == "few":
        score = (i * 2654435761 % 5).float()
    elif kind == "zeros":
        score = torch.where(i % 3 == 0, -0.0, 0.0)
    elif kind == "nan":
        score[i % 3 > 0] = float("nan")
        score[i % 7 == 0] = -float("nan")
    elif kind == "inf":
        score[i % 5 == 0] = float("inf")
        score[i % 5 == 1] = -float("inf")
    elif kind == "negative":
        score = -score
    elif kind == "rising":
        score = i.float()
    else:
        score = -i.float()
    for keep, sink, recent in ((2500, 4, 64), (4999, 0, 0), (10, 5, 5), (11, 5, 5)):
        run(kv, score, [n, n], off, at, [keep, keep - 1 if sink == 0 else keep], sink, recent, 2, dst=dst)


@gpu
@pytest.mark.parametrize("dst", [False, True])
def test_many_layers(dst):
    lens = [900, 1200, 333]
    kv, score, off, at = make(lens, 61, 576, torch.bfloat16, 6)
    run(kv, score, lens, off, at, [512, 512, 512], 4, 128, 61, dst=dst)


@gpu
def test_statuses_and_skipped_requests():
    lens, layers = [100, 50, 80, 60, 90], 2
    kv, score, off, at = make(lens, layers, 16, torch.float32, 1)
    i32 = dict(dtype=torch.int32, device=DEV)
    cl = torch.tensor(lens, **i32)
    offs = torch.tensor(off, device=DEV)
    offs[1] = at - 49                                         # on the last layer it ends one row behind the pool
    keep = torch.tensor([40, 20, 9, 70, -1], **i32)           # request 2: less than sink + recent; 3: all stay; 4: negative
    dkv, dscore = kv.to(DEV), score.to(DEV)
    status = torch.full((5,), 9, **i32)
    out = lib.cache_evict(dkv, dscore, offs, cl, keep, 4, 6, 100, n_layers=layers, layer_stride_rows=at, max_keep=65,
                          status=status)
    assert status.tolist() == [lib.DDT_OK, lib.DDT_ERR_BOUNDS, lib.DDT_ERR_INPUT, lib.DDT_OK, lib.DDT_ERR_INPUT]
    assert cl.tolist() == [40, 50, 80, 60, 90] and out["new_len"] is cl
    assert bool((out["src"][:, [1, 2, 4]] == -1).all())
    same = torch.ones(layers * at, dtype=torch.bool)
    for la in range(layers):
        same[la * at + off[0]:la * at + off[0] + 100] = False
    assert torch.equal(dkv.cpu()[same], kv[same]) and torch.equal(dscore.cpu()[same], score[same])
    # a list too short for the kept rows, and destinations outside their pool
    cl = torch.tensor(lens, **i32)
    keep = torch.full((5,), 30, **i32)
    d2 = {"kv": torch.zeros(100, 16, device=DEV), "score": torch.zeros(100, device=DEV),
          "off": torch.tensor([0, 71, 40, -1, 70], device=DEV), "layer_stride_rows": 0}
    out = lib.cache_evict(kv.to(DEV), score.to(DEV), torch.tensor(off, device=DEV), cl, keep, 4, 6, 100, dst=d2,
                          max_keep=64, status=status)
    assert status.tolist() == [0, lib.DDT_ERR_BOUNDS, 0, lib.DDT_ERR_BOUNDS, 0]
    assert out["new_len"].tolist() == [30, 0, 30, 0, 30]
    out = lib.cache_evict(kv.to(DEV), score.to(DEV), torch.tensor(off, device=DEV), cl, keep, 4, 6, 100, max_keep=29,
                          status=status)
    assert status.tolist() == [lib.DDT_ERR_CAPACITY] * 5 and cl.tolist() == lens


@gpu
def test_offsets_at_the_64_bit_limit_are_out_of_bounds():
    kv, score, off, at = make([100, 100, 100], 2, 16, torch.float32, 1)
    i32 = dict(dtype=torch.int32, device=DEV)
    offs = torch.tensor([2 ** 63 - 1, off[1], 2 ** 63 - 60], device=DEV)
    cl, status = torch.tensor([100] * 3, **i32), torch.full((3,), 9, **i32)
    dkv = kv.to(DEV)
    lib.cache_evict(dkv, score.to(DEV), offs, cl, torch.tensor([50] * 3, **i32), 4, 6, 100, n_layers=2,
                    layer_stride_rows=at, status=status)
    assert status.tolist() == [lib.DDT_ERR_BOUNDS, 0, lib.DDT_ERR_BOUNDS] and cl.tolist() == [100, 50, 100]
    for la in range(2):
        assert torch.equal(dkv[la * at + off[0]:la * at + off[0] + 100].cpu(), kv[la * at + off[0]:la * at + off[0] + 100])
    d2 = {"kv": torch.zeros(400, 16, device=DEV), "score": torch.zeros(400, device=DEV),
          "off": torch.tensor([0, 2 ** 63 - 10, 100], device=DEV), "layer_stride_rows": 200}
    cl = torch.tensor([100] * 3, **i32)
    out = lib.cache_evict(kv.to(DEV), score.to(DEV), torch.tensor(off, device=DEV), cl, torch.tensor([50] * 3, **i32), 4, 6,
                          100, n_layers=2, layer_stride_rows=at, dst=d2, status=status)
    assert status.tolist() == [0, lib.DDT_ERR_BOUNDS, 0] and out["new_len"].tolist() == [50, 0, 50]


@gpu
@pytest.mark.parametrize("dst", [False, True])
@pytest.mark.parametrize("B,layers,n", [(1, 1, 40001), (2, 8, 20001), (5, 7, 12011), (7, 8, 11003), (16, 4, 9001), (3, 61, 2050)])
def test_cluster_splits(B, layers, n, dst):
    """From one request over eight CTAs to one CTA per layer and request."""
    lens = [max(1, n - 700 * b) if b % 4 else n for b in range(B)]
    kv, score, off, at = make(lens, layers, 24, torch.bfloat16, B * layers)
    score[torch.arange(score.numel()) % 3 == 0] = 0.75  # ties across the slices
    run(kv, score, lens, off, at, [n // 3 + 1] * B, 3, 100, layers, dst=dst)


@gpu
def test_one_pool_holds_source_and_destination():
    """A request moves into a free region of the same pool."""
    kv, score, off, at = make([400], 2, 32, torch.float32, 2)
    pool = torch.cat([kv.view(2, at, 32), torch.zeros(2, 200, 32)], 1).reshape(-1, 32).to(DEV)
    sc = torch.cat([score.view(2, at), torch.zeros(2, 200)], 1).reshape(-1).to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    d2 = {"kv": pool.view(-1, 32)[1:], "score": sc[1:], "off": torch.tensor([at], device=DEV), "layer_stride_rows": at + 200}
    lib.cache_evict(pool, sc, torch.tensor(off, device=DEV), torch.tensor([400], **i32), torch.tensor([150], **i32), 2, 30,
                    400, n_layers=2, layer_stride_rows=at + 200, dst=d2)
    for la in range(2):
        idx = kept_rows(score[la * at + off[0]:la * at + off[0] + 400].numpy(), 150, 2, 30)
        to = la * (at + 200) + at + 1
        assert torch.equal(pool[to:to + 150].cpu(), kv[la * at + off[0] + torch.from_numpy(idx)])


@gpu
def test_rows_beyond_32_bit_offsets():
    """Row bytes whose offset passes 2^32, element offsets past 2^31."""
    rows, d = 4_000_000, 576
    kv = torch.zeros(rows, d, dtype=torch.bfloat16, device=DEV)
    score = torch.zeros(rows, device=DEV)
    off, n = rows - 5000, 5000
    g = torch.Generator(device=DEV).manual_seed(1)
    kv[off:] = torch.randn(n, d, device=DEV, generator=g).bfloat16()
    score[off:] = torch.rand(n, device=DEV, generator=g)
    idx = torch.from_numpy(kept_rows(score[off:].cpu().numpy(), 2000, 4, 100)).to(DEV)
    ref = kv[off:][idx].clone()
    cl = torch.tensor([n], dtype=torch.int32, device=DEV)
    lib.cache_evict(kv, score, torch.tensor([off], device=DEV), cl, torch.tensor([2000], dtype=torch.int32, device=DEV), 4,
                    100, n)
    assert torch.equal(kv[off:off + 2000], ref) and cl.tolist() == [2000]


@gpu
def test_replayed_graph_and_side_stream():
    lens = [700, 900]
    kv, score, off, at = make(lens, 2, 64, torch.float32, 9)
    i32 = dict(dtype=torch.int32, device=DEV)
    a = dict(kv=kv.to(DEV), score=score.to(DEV))
    offs, keep = torch.tensor(off, device=DEV), torch.tensor([300, 300], **i32)
    cl = torch.tensor(lens, **i32)
    ws = torch.empty(lib.cache_evict_workspace_size(2, 2, 900), dtype=torch.uint8, device=DEV)
    out = {"src": torch.empty(2, 2, 900, **i32), "new_len": cl}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.cache_evict(a["kv"], a["score"], offs, cl, keep, 4, 32, 900, n_layers=2, layer_stride_rows=at, out=out,
                        workspace=ws)
    for r in range(2):  # fresh rows and lengths under the same graph
        sc = torch.rand(2 * at, generator=torch.Generator().manual_seed(r))
        a["kv"].copy_(kv)
        a["score"].copy_(sc)
        cl.copy_(torch.tensor(lens, **i32))
        g.replay()
        torch.cuda.synchronize()
        for b in range(2):
            idx = kept_rows(sc[at + off[b]:at + off[b] + lens[b]].numpy(), 300, 4, 32)
            assert torch.equal(a["kv"][at + off[b]:at + off[b] + 300].cpu(), kv[at + off[b] + torch.from_numpy(idx)])
        assert cl.tolist() == [300, 300]
    side = torch.cuda.Stream()
    cl2 = torch.tensor(lens, **i32)
    k2, s2 = kv.to(DEV), score.to(DEV)
    side.wait_stream(torch.cuda.current_stream())
    lib.cache_evict(k2, s2, offs, cl2, keep, 4, 32, 900, n_layers=2, layer_stride_rows=at, stream=side)
    side.synchronize()
    idx = kept_rows(score[off[0]:off[0] + 700].numpy(), 300, 4, 32)
    assert torch.equal(k2[off[0]:off[0] + 300].cpu(), kv[off[0] + torch.from_numpy(idx)])


@gpu
def test_bindings_refusals():
    kv, score, off, at = make([50], 1, 16, torch.float32, 1)
    i32 = dict(dtype=torch.int32, device=DEV)
    a = [kv.to(DEV), score.to(DEV), torch.tensor(off, device=DEV), torch.tensor([50], **i32), torch.tensor([20], **i32), 0, 0,
         50]
    with pytest.raises(ValueError):
        lib.cache_evict(kv, *a[1:])
    with pytest.raises(ValueError):
        lib.cache_evict(a[0], a[1][:-1], *a[2:])
    with pytest.raises(TypeError):
        lib.cache_evict(a[0].half(), *a[1:])
    with pytest.raises(TypeError):
        lib.cache_evict(*a[:3], a[3].long(), *a[4:])
    with pytest.raises(ValueError):
        lib.cache_evict(*a, out={"new_len": a[3]})
    with pytest.raises(lib.DDTError):
        lib.cache_evict(*a[:5], -1, 0, 50)
    with pytest.raises(lib.DDTError):
        lib.cache_evict(*a, n_layers=2)
    with pytest.raises(lib.DDTError):  # a destination that is the source pool's first row
        lib.cache_evict(*a, dst={"kv": a[0], "score": a[1], "off": a[2]})


def test_host_validation():
    build.build()
    so = lib.load()
    p = ctypes.c_void_p(256)
    q = ctypes.c_void_p(1 << 20)
    assert lib.cache_evict_workspace_size(4, 61, 1000) >= 4 * 61 * 8
    assert lib.cache_evict_workspace_size(0, 1, 10) == 0

    def call(kv=p, dtype=1, d=576, score=p, layers=1, stride=100, sink=0, recent=0, B=2, ml=50, kd=None, rows=0, sd=None, ds=0,
             od=None, nl=p, src=p, mk=50, ws=p, wsb=1 << 16):
        return so.ddt_cache_evict(kv, 100, dtype, d, score, layers, stride, p, p, p, sink, recent, B, ml, kd, rows, sd, ds, od,
                                  nl, src, mk, None, ws, wsb, None)

    bad = lib.DDT_ERR_INVALID_ARG
    assert call(kv=None) == call(score=None) == call(nl=None) == call(src=None) == call(ws=None) == bad
    assert call(dtype=3) == call(d=0) == call(d=1) == call(B=0) == call(layers=0) == call(mk=0) == call(ml=-1) == bad
    assert call(layers=2, stride=0) == call(sink=-1) == call(recent=-1) == call(wsb=8) == bad
    assert call(ws=ctypes.c_void_p(128)) == call(kv=ctypes.c_void_p(258)) == bad
    assert call(kd=q) == call(kd=q, sd=q) == call(od=q) == call(kd=p, sd=q, od=q, rows=5) == call(kd=q, sd=q, od=q) == bad
    assert call(layers=2, kd=q, sd=q, od=q, rows=5) == bad  # no destination layer stride
    assert call(mk=(1 << 30) + 1) == bad                    # row numbers past 32 bits
    assert call(layers=3, stride=1 << 62) == bad            # a stride that no pool can have
    assert call(layers=3, kd=q, sd=q, od=q, rows=5, ds=1 << 62) == bad
