"""ddt_token_logprobs against the definition in 64 bits: log-probs of given
tokens, entropy and top alternatives, on vocabularies from one token to many,
rows that are not aligned or padded, masked logits (-inf, the type's lowest
value), rows of equal values, rising rows, node lists with skipped entries,
and entries that must be reported."""
import ctypes

import numpy as np
import pytest
import torch

from ddtree_speculative_decode_b200 import build, lib

DEV = "cuda:0"
gpu = pytest.mark.gpu

# The kernel's sums are float32: s = sum e^(x - m) and u = sum e^(x - m)(x - m)
# over at most 2^18 terms. A thread adds at most 2^11 terms in sequence to one
# of two accumulators and the rest joins in trees, so a sum of n rounded terms
# is off by at most (2^10 + 40) 2^-24 relative to the sum of magnitudes in the
# worst case and by about sqrt of that count in practice; the terms themselves
# carry the exponential's 2^-22 plus the exponent's rounding |y| 2^-23. With
# |x - m| <= 60 for every term that matters: 2^-22 + 60 2^-23 < 8e-6 worst
# case per term, 1e-6 typical after averaging. ln s moves by the relative
# error of s; the entropy by that plus |u / s| times it (|u / s| <= 60).
# Bounds used: logp 1e-5 + 2^-23 |logp|; entropy 2e-5 + 2e-6 |H|.
LOGP_ABS, LOGP_REL = 1e-5, 2.0 ** -22
ENT_ABS, ENT_REL = 2e-5, 2e-6


def reference(x, tok, nodes, K):
    """x [B, N, V] float64 on any device, tok / nodes [B, M] int64."""
    B, N, V = x.shape
    M = tok.shape[1]
    logp = torch.zeros(B, M, dtype=torch.float64)
    ent = torch.zeros(B, M, dtype=torch.float64)
    tl = torch.full((B, M, K), -np.inf, dtype=torch.float64)
    tt = torch.full((B, M, K), -1, dtype=torch.int64)
    st = torch.zeros(B, M, dtype=torch.int64)
    for b in range(B):
        for j in range(M):
            i = int(nodes[b, j])
            if i < 0:
                continue
            t = int(tok[b, j])
            row = x[b, i] if i < N else None
            if row is None or not 0 <= t < V or bool(torch.isnan(row).any()) or float(row.max()) in (np.inf, -np.inf):
                logp[b, j], st[b, j] = -np.inf, lib.DDT_ERR_INPUT
                continue
            y = row - row.max()
            lz = torch.log(torch.exp(y).sum())
            lp = y - lz
            logp[b, j] = lp[t]
            p = torch.exp(lp)
            ent[b, j] = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum()
            if K:
                order = torch.sort(row, descending=True, stable=True).indices[:K]
                n = min(K, int(torch.isfinite(row).sum()))
                tl[b, j, :n] = lp[order[:n]].cpu()
                tt[b, j, :n] = order[:n].cpu()
    return {"logp": logp, "entropy": ent, "top_logp": tl, "top_tok": tt, "status": st}


def close(got, ref, a, r):
    got = got.double().cpu()
    # the outputs are float32: a log-prob beyond -3.4e38 (a gap of twice the lowest value) rounds to -inf
    ref = torch.where(ref.abs() > torch.finfo(torch.float32).max, torch.sign(ref) * np.inf, ref)
    fin = torch.isfinite(ref)
    assert torch.equal(fin, torch.isfinite(got)) and torch.equal(got[~fin], ref[~fin])
    d = (got[fin] - ref[fin]).abs()
    assert bool((d <= a + r * ref[fin].abs()).all()), float(d.max())


def check(logits, tok, nodes=None, K=0, **kw):
    B, N, V = logits.shape
    M = tok.shape[1]
    dn = None if nodes is None else nodes.to(DEV, torch.int32)
    out = lib.token_logprobs(logits, tok.to(DEV, torch.int32), nodes=dn, K=K, **kw)
    torch.cuda.synchronize()
    full = torch.arange(M).expand(B, M) if nodes is None else nodes
    ref = reference(logits.double(), tok.long(), full.long(), K)
    assert torch.equal(out["status"].cpu().long(), ref["status"])
    assert torch.equal(out["top_tok"].cpu().long(), ref["top_tok"])
    close(out["logp"], ref["logp"], LOGP_ABS, LOGP_REL)
    close(out["entropy"], ref["entropy"], ENT_ABS, ENT_REL)
    close(out["top_logp"], ref["top_logp"], LOGP_ABS, LOGP_REL)
    return out


def make(B, N, V, dtype, seed, sigma=3.0, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    full = torch.randn(B, N, V + pad, device=DEV, generator=g).mul_(sigma).to(dtype)
    tok = torch.randint(0, V, (B, N), device=DEV, generator=g)
    return full[:, :, :V], tok.cpu()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,K", [(1, 1), (2, 0), (3, 3), (7, 5), (8, 8), (9, 4), (255, 32), (1001, 0), (1024, 1), (4099, 7),
                                 (8192, 32), (16384, 16), (32003, 8), (65537, 20), (163840, 8), (163841, 32)])
def test_vocabularies(V, K, dtype):
    logits, tok = make(2, 3, V, dtype, V + K)
    check(logits, tok, K=K)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [1, 3, 8, 21])
def test_padded_rows_and_every_alignment(pad, dtype):
    logits, tok = make(3, 9, 5000 + pad, dtype, pad, pad=pad)
    logits[:] = logits
    check(logits, tok, K=5)
    check(logits[1:2, 2:3], tok[1:2, 2:3].contiguous(), K=3)  # one row that starts anywhere


@gpu
@pytest.mark.parametrize("B,N", [(1, 1), (1, 130), (5, 33), (37, 16), (700, 1), (3, 1500)])
def test_row_counts(B, N):
    """From one row for the whole grid to several rounds of rows, with C = 8 .. 1 CTAs per row."""
    logits, tok = make(B, N, 20011, torch.bfloat16, B + N)
    check(logits, tok, K=6)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [0, 1, 8, 32])
def test_masked_logits(K, dtype):
    lowest = torch.finfo(dtype).min
    logits, tok = make(1, 8, 30000, dtype, 5)
    logits[0, 0, 100:] = -np.inf
    logits[0, 1, ::2] = -np.inf
    logits[0, 2] = -np.inf
    logits[0, 2, 12345] = 1.5                  # one possible token
    tok[0, 2] = 12345
    logits[0, 3, 3:] = lowest
    logits[0, 4] = lowest                      # every token equally unlikely
    logits[0, 5] = -np.inf
    logits[0, 5, 7] = lowest                   # the lowest value is still the only token
    tok[0, 5] = 7
    logits[0, 6, 1:] = lowest
    logits[0, 6, 0] = -lowest                  # the largest finite value
    logits[0, 7] = -np.inf                     # nothing possible: reported
    check(logits, tok, K=K)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,V,K", [(1, 50021, 32), (30, 50021, 9), (60, 33000, 20), (1, 163840, 8), (2, 9001, 2)])
def test_where_the_largest_values_lie(B, V, K, dtype):
    """The alternatives side by side, a round of vectors apart, at the row's ends, or all but one of them apart from it."""
    logits, tok = make(B, 9, V, dtype, V + B)
    high = torch.linspace(16, 31.5, K, device=DEV)
    logits[:, 0, 1000:1000 + K] = high
    step = V // K // 1024 * 1024 or V // K
    logits[:, 1, 17:17 + step * (K - 1) + 1:step] = high
    logits[:, 2, :K] = high
    logits[:, 3, V - K:] = high.flip(0)
    logits[:, 4, 5000:5300] = 20.0                   # more equal values than are listed
    logits[:, 5, :8] = 20.0                          # and fewer
    logits[:, 6, 2048:2048 + 8 * K:8] = high         # one per vector of a warp
    logits[:, 7, V // 2] = 30.0
    logits[:, 8, ::V // 150] = 20.0                  # equal ones, spread
    check(logits, tok, K=K)


@gpu
@pytest.mark.parametrize("K", [1, 5, 32])
@pytest.mark.parametrize("V", [40000, 163840])
def test_ties_and_order(V, K):
    """Rows in which far more than K values reach any bound of the first loads."""
    logits = torch.empty(1, 8, V, device=DEV)
    logits[0, 0] = 0.25                                             # all equal: the lowest tokens
    logits[0, 1] = torch.arange(V, device=DEV) * 1e-3               # rising
    logits[0, 2] = -torch.arange(V, device=DEV) * 1e-3              # falling
    logits[0, 3] = (torch.arange(V, device=DEV) % 7).float()        # few distinct values
    logits[0, 4] = (torch.arange(V, device=DEV) // 4096).float()    # steps
    logits[0, 5] = torch.where(torch.arange(V, device=DEV) >= V - 3, 5.0, -0.0)
    logits[0, 6] = torch.where(torch.arange(V, device=DEV) % 2 == 0, 0.0, -0.0)  # equal zeros
    logits[0, 7] = torch.randint(0, 3, (V,), device=DEV).float()
    tok = torch.tensor([[0, V - 1, 5, 6, V // 2, V - 1, 3, 2]])
    check(logits, tok, K=K)
    check(logits.bfloat16(), tok, K=K)


@gpu
@pytest.mark.parametrize("K", [0, 4])
def test_reported_rows(K):
    logits, tok = make(2, 5, 9000, torch.float32, 3)
    logits[0, 0, 8999] = np.nan
    logits[0, 1, 0] = np.inf
    logits[1, 2, 4000] = -np.nan
    tok[0, 3] = 9000
    tok[0, 4] = -1
    nodes = torch.arange(5).repeat(2, 1)
    nodes[1, 4] = 5
    check(logits, tok, nodes, K=K)


@gpu
@pytest.mark.parametrize("B,N,M", [(1, 64, 64), (4, 16, 16), (3, 1, 5), (2, 300, 7), (9, 40, 1000)])
def test_node_lists(B, N, M):
    """Skipped entries anywhere, the same node more than once, more entries than rows, several launches."""
    logits, _ = make(B, N, 3000, torch.bfloat16, M)
    g = torch.Generator().manual_seed(B * N + M)
    nodes = torch.randint(-N, N, (B, M), generator=g)
    tok = torch.randint(0, 3000, (B, M), generator=g)
    tok[nodes < 0] = -7
    check(logits, tok, nodes, K=3)


@gpu
def test_nothing_selected():
    logits, tok = make(2, 4, 500, torch.float32, 1)
    check(logits, tok, torch.full((2, 4), -1), K=2)


@gpu
def test_unread_rows_do_not_matter():
    logits, tok = make(1, 6, 7001, torch.float32, 2)
    nodes = torch.tensor([[4, -1, 2, -1, -1, -1]])
    logits[0, [0, 1, 3, 5]] = np.nan
    check(logits, tok, nodes, K=2)


@gpu
def test_offsets_beyond_32_bits():
    """Rows whose element offset passes 2^31."""
    N, V = 14000, 163840
    logits = torch.zeros(1, N, V, dtype=torch.bfloat16, device=DEV)
    rows = torch.tensor([0, 13107, 13108, 13999])
    g = torch.Generator(device=DEV).manual_seed(9)
    for r in rows.tolist():
        logits[0, r] = torch.randn(V, device=DEV, generator=g).bfloat16()
    tok = torch.tensor([[1, 2, 163839, 77]])
    out = lib.token_logprobs(logits, tok.to(DEV, torch.int32), nodes=rows[None].to(DEV, torch.int32), K=3)
    ref = reference(logits[:, rows.to(DEV)].double(), tok, torch.arange(4)[None], 3)
    assert torch.equal(out["top_tok"].cpu().long(), ref["top_tok"])
    close(out["logp"], ref["logp"], LOGP_ABS, LOGP_REL)


@gpu
def test_repeats_streams_and_graphs():
    """The same call gives the same bits, on another stream and replayed from a graph with new inputs."""
    logits, tok = make(2, 40, 50001, torch.bfloat16, 8)
    tok = tok.to(DEV, torch.int32)
    ref = {k: v.clone() for k, v in lib.token_logprobs(logits, tok, K=8).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lib.token_logprobs(logits, tok, K=8, stream=side)
    side.synchronize()
    for k in ref:
        assert torch.equal(got[k], ref[k]), k
    out = lib.alloc_logprobs(2, 40, 8, DEV)
    other, _ = make(2, 40, 50001, torch.bfloat16, 9)
    held = other.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.token_logprobs(held, tok, K=8, out=out)
    held.copy_(logits)
    g.replay()
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(out[k], ref[k]), k


@gpu
def test_bindings_refusals():
    logits, tok = make(2, 4, 100, torch.float32, 1)
    t = tok.to(DEV, torch.int32)
    with pytest.raises(ValueError):
        lib.token_logprobs(logits.cpu(), t)
    with pytest.raises(TypeError):
        lib.token_logprobs(logits.half(), t)
    with pytest.raises(TypeError):
        lib.token_logprobs(logits, t.long())
    with pytest.raises(ValueError):
        lib.token_logprobs(logits.transpose(1, 2), t)          # rows not contiguous
    with pytest.raises(ValueError):
        lib.token_logprobs(logits[:, :3], t[:, :3].contiguous())  # rows not evenly spaced
    with pytest.raises(ValueError):
        lib.token_logprobs(logits, t, nodes=t[:1])
    with pytest.raises(lib.DDTError):
        lib.token_logprobs(logits, t, K=33)
    with pytest.raises(lib.DDTError):
        lib.token_logprobs(logits, torch.zeros(2, 5, dtype=torch.int32, device=DEV))  # M > N without nodes


def test_host_validation():
    build.build()
    so = lib.load()
    p = ctypes.c_void_p(256)

    def call(logits=p, dtype=1, V=100, stride=100, nodes=p, tok=p, B=2, N=4, M=4, K=2, logp=p, top=p):
        return so.ddt_token_logprobs(logits, dtype, V, stride, nodes, tok, B, N, M, K, logp, None, top, top, None, None)

    bad = lib.DDT_ERR_INVALID_ARG
    assert call(logits=None) == call(tok=None) == call(logp=None) == call(top=None) == bad
    assert call(V=0) == call(B=0) == call(N=0) == call(M=0) == call(stride=99) == call(dtype=5) == bad
    assert call(K=-1) == call(K=33) == call(V=1, K=2) == call(nodes=None, M=5) == bad
    assert call(logits=ctypes.c_void_p(257)) == bad                      # not aligned to the element
    assert call(B=1 << 20, M=1 << 12) == lib.DDT_ERR_UNSUPPORTED
    assert call(V=(1 << 30) + 1, stride=1 << 31) == lib.DDT_ERR_UNSUPPORTED
