"""Cases of the cache-budget and token-scoring operators, with their plain forms.

Three operators around a verify step of speculative decoding:

- ``logprobs``: log probabilities of given tokens at verify rows, the rows' entropy and their top alternatives;
- ``weights``: the attention weight every cached row received from selected verify rows, accumulated per row;
- ``evict``: the first, the last and the best-scored rows of every request's cache move, in order, into another region.

``run`` computes them in elementary torch operations, or, where ``own`` is true, through the library's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
NEG_INF = float("-inf")


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------


def _logprobs(B, N, V, dtype, path, K, masked=0.0, pad=0):
    """path: accepted nodes per request at most (0: every verify row). masked: share of tokens at -inf. pad: unused
    columns behind the vocabulary."""
    return {"op": "logprobs", "B": B, "N": N, "V": V, "dtype": dtype, "path": path, "K": K, "masked": masked, "pad": pad}


def _weights(B, N, H, d, lo, hi, dtype, path, kv_scale, scale, decay):
    """lo, hi: range of the requests' cache lengths. path: nodes on the accepted path at most, causal among themselves
    (0: every verify row, each seeing the whole cache)."""
    return {"op": "weights", "B": B, "N": N, "H": H, "d": d, "lo": lo, "hi": hi, "dtype": dtype, "path": path,
            "kv_scale": kv_scale, "scale": scale, "decay": decay}


def _evict(B, layers, d, lo, hi, keep, sink, recent, dtype):
    return {"op": "evict", "B": B, "layers": layers, "d": d, "lo": lo, "hi": hi, "keep": keep, "sink": sink,
            "recent": recent, "dtype": dtype}


MLA = 1 / math.sqrt(192)  # the softmax scale of 128 + 64 dims per head


def listed():
    named = [
        # the answer's logprobs of one request's accepted path: the smallest call, latency
        ("logprobs path 1req", _logprobs(1, 64, 163840, "bf16", 8, 0)),
        # every verify row of the long-context step, with alternatives, tokens masked by a grammar
        ("logprobs rows 4req", _logprobs(4, 128, 163840, "bf16", 0, 8, masked=0.3)),
        # float32 logits, odd vocabulary, rows that are not 16-byte aligned
        ("logprobs f32 odd", _logprobs(3, 33, 50021, "f32", 0, 20, pad=3)),
        # scoring of whole texts: a large batch of rows with the best alternative
        ("logprobs rows 64req", _logprobs(64, 64, 163840, "bf16", 0, 1)),
        # one decoded token of one request: the smallest cache call
        ("weights token 1req", _weights(1, 1, 64, 576, 4096, 4096, "bf16", 0, 0.1, MLA, 1.0)),
        # the accepted path of a 64-node tree
        ("weights path 1req", _weights(1, 64, 64, 576, 4096, 4096, "bf16", 9, 0.1, MLA, 0.98)),
        # single-token serving of a ragged batch
        ("weights token 16req", _weights(16, 1, 64, 576, 1024, 8192, "bf16", 0, 1.0, MLA, 1.0)),
        # every row of the long-context trees: the largest
        ("weights tree 4req", _weights(4, 128, 64, 576, 32768, 32768, "bf16", 0, 0.1, MLA, 1.0)),
        # the float32 path at the tiny model's heads and dims, longer cache
        ("weights f32 small", _weights(4, 8, 4, 80, 300, 2000, "f32", 5, 1.0, 1 / math.sqrt(24), 0.9)),
        # one layer of one request halved: latency of the selection
        ("evict 1req", _evict(1, 1, 576, 4096, 4096, 2048, 4, 256, "bf16")),
        # a ragged batch, some requests under their budget already
        ("evict 16req", _evict(16, 4, 576, 1024, 8192, 2048, 4, 512, "bf16")),
        # long contexts halved on many layers: the rows' copy
        ("evict 4req long", _evict(4, 16, 576, 32768, 32768, 16384, 4, 1024, "bf16")),
    ]
    return [dict(c, name=name) for name, c in named]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("logprobs", "weights", "evict"))
    if op == "logprobs":
        V = rng.choice((163840, _log(rng, 400, 200000)))
        N = _log(rng, 1, 256)
        B = _log(rng, 1, max(1, min(64, int(4e8 / (V * N)))))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        return _logprobs(B, N, V, dtype, rng.choice((0, 0, min(N, 16))), rng.choice((0, 1, 5, 8, 20, 32)),
                         masked=rng.choice((0.0, 0.0, 0.5)), pad=rng.choice((0, 0, 1, 24)))
    if op == "weights":
        if rng.random() < 0.25:
            N = _log(rng, 1, 32)
            return _weights(_log(rng, 1, 8), N, rng.choice((2, 4, 7)), rng.choice((40, 80, 96)), 1, _log(rng, 2, 3000), "f32",
                            rng.choice((0, min(N, 6))), 1.0, 0.2, rng.choice((1.0, 0.9)))
        N, B, hi = _log(rng, 1, 128), _log(rng, 1, 32), _log(rng, 64, 60000)
        while B * N * hi > 8000000:
            B, N, hi = max(1, B // 2), max(1, N // 2), max(64, hi * 3 // 4)
        return _weights(B, N, rng.choice((8, 16, 64, 64, 64, 128)), 576, max(1, hi // 4), hi, "bf16",
                        rng.choice((0, min(N, 9))), rng.choice((0.1, 1.0)), MLA, rng.choice((1.0, 0.98)))
    B, hi = _log(rng, 1, 32), _log(rng, 200, 60000)
    layers = _log(rng, 1, max(1, min(61, int(1800000 / (B * hi)))))
    while B * hi * layers > 2000000:
        B = max(1, B // 2)
    keep = max(2, int(hi * rng.uniform(0.1, 0.9)))
    sink = min(keep // 2, rng.choice((0, 1, 4)))
    return _evict(B, layers, rng.choice((576, 576, 80)), max(1, hi // 5), hi, keep, sink,
                  min(keep - sink, int(keep * rng.uniform(0, 0.5))), rng.choice(("bf16", "bf16", "f32")))


def _lens(case):
    """The requests' cache lengths: fixed by the case, so that work() can count them."""
    r = random.Random(case["B"] * 1000003 + case["hi"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _paths(case):
    """The accepted path's length of every request, or None."""
    if not case["path"]:
        return None
    r = random.Random(case["B"] * 7919 + case["N"])
    return [r.randint(max(1, case["path"] // 2), case["path"]) for _ in range(case["B"])]


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gen(seed, salt):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 16 + salt)


def _normal(shape, dtype, gen, scale=1.0):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, scale, generator=gen)


def _node_lists(case, paths, seed):
    """[B, N] ascending node indices from the root, then -1, as the accept walk writes them."""
    r = random.Random(int(seed))
    rows = [[0] + sorted(r.sample(range(1, case["N"]), m - 1)) + [-1] * (case["N"] - m) for m in paths]
    return torch.tensor(rows, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    return {"logprobs": _prepare_logprobs, "weights": _prepare_weights, "evict": _prepare_evict}[case["op"]](case, seed)


def _prepare_logprobs(case, seed):
    B, N, V, gen = case["B"], case["N"], case["V"], _gen(seed, 1)
    full = _normal((B, N, V + case["pad"]), _dtype(case), gen, 3.0)
    logits = full[:, :, :V]
    if case["masked"]:
        banned = torch.rand(V, device=DEV, generator=gen) < case["masked"]
        logits.masked_fill_(banned, NEG_INF)
    paths = _paths(case)
    nodes = None if paths is None else _node_lists(case, paths, seed)
    tok = torch.randint(0, V, (B, N), dtype=torch.int32, device=DEV, generator=gen)
    greedy = torch.stack([r.argmax(-1) for r in logits]).to(torch.int32)  # most given tokens are the greedy ones
    at = torch.arange(N, device=DEV).expand(B, N) if nodes is None else nodes.clamp_min(0).long()
    tok = torch.where(torch.rand((B, N), device=DEV, generator=gen) < 0.8, greedy.gather(1, at), tok)
    if nodes is not None:
        tok = torch.where(nodes < 0, torch.full_like(tok, -1), tok)
    return {"case": case, "logits": logits, "nodes": nodes, "tok": tok.contiguous()}


def _pool(case, layers=1):
    """(lengths, offsets, rows of one layer): requests one behind the other, a few rows apart."""
    lens, off, at = _lens(case), [], 0
    for n in lens:
        off.append(at)
        at += n + 5
    return lens, off, at


def _prepare_weights(case, seed):
    B, N, H, d, gen = case["B"], case["N"], case["H"], case["d"], _gen(seed, 2)
    lens, off, rows = _pool(case)
    kv = _normal((rows, d), _dtype(case), gen, case["kv_scale"])
    q = _normal((B, N, H, d), _dtype(case), gen)
    paths = _paths(case)
    nodes = None if paths is None else _node_lists(case, paths, seed)
    lse = torch.empty((B, N, H), dtype=torch.float32, device=DEV)
    for b in range(B):  # what the verify attention gave for these rows, over the whole cache
        k = kv[off[b]:off[b] + lens[b]].float()
        for i in range(0, N, 16):
            lse[b, i:i + 16] = torch.logsumexp(case["scale"] * (q[b, i:i + 16].float() @ k.T), -1)
    prev = torch.empty(rows, dtype=torch.float32, device=DEV).exponential_(1.0, generator=gen)
    return {"case": case, "q": q, "kv": kv, "lse": lse, "nodes": nodes, "prev": prev, "score": torch.zeros_like(prev),
            "off": torch.tensor(off, dtype=torch.int64, device=DEV), "len": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "n": torch.full((B,), N, dtype=torch.int32, device=DEV)}


def _prepare_evict(case, seed):
    B, layers, d, gen = case["B"], case["layers"], case["d"], _gen(seed, 3)
    lens, off, rows = _pool(case)
    kept = [min(n, case["keep"]) for n in lens]
    dst_off, dst_rows = [], 0
    for n in kept:
        dst_off.append(dst_rows)
        dst_rows += n + 3
    kv = _normal((layers * rows, d), _dtype(case), gen, 0.1)
    score = _normal((layers * rows,), torch.float32, gen, 2.0).exp_()
    score[torch.rand(layers * rows, device=DEV, generator=gen) < 0.05] = 0.0  # rows that nothing attended to: ties
    return {"case": case, "kv": kv, "score": score, "rows": rows, "dst_rows": dst_rows,
            "off": torch.tensor(off, dtype=torch.int64, device=DEV), "len": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "keep": torch.full((B,), case["keep"], dtype=torch.int32, device=DEV),
            "dst_off": torch.tensor(dst_off, dtype=torch.int64, device=DEV),
            "dst_kv": torch.zeros((layers * dst_rows, d), dtype=_dtype(case), device=DEV),
            "dst_score": torch.zeros(layers * dst_rows, dtype=torch.float32, device=DEV),
            "src": torch.full((layers, B, case["keep"]), -1, dtype=torch.int32, device=DEV),
            "new_len": torch.zeros(B, dtype=torch.int32, device=DEV),
            "lens": lens, "offs": off, "dst_offs": dst_off}


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------


def run(state):
    return {"logprobs": _run_logprobs, "weights": _run_weights, "evict": _run_evict}[state["case"]["op"]](state)


def _run_logprobs(s):
    case = s["case"]
    K = case["K"]
    if own:
        from ddtree_speculative_decode_b200 import lib
        if "out" not in s:
            s["out"] = lib.alloc_logprobs(s["tok"].shape[0], s["tok"].shape[1], K, s["tok"].device)
        out = lib.token_logprobs(s["logits"], s["tok"], nodes=s["nodes"], K=K, out=s["out"])
        return {k: out[k] for k in ("logp", "entropy") + (("top_logp", "top_tok") if K else ())}
    B, N, V = s["logits"].shape
    M = s["tok"].shape[1]
    nodes = torch.arange(M, dtype=torch.int32, device=DEV).expand(B, M) if s["nodes"] is None else s["nodes"]
    live = (nodes >= 0).reshape(-1)
    row = (torch.arange(B, device=DEV)[:, None] * N + nodes.clamp_min(0)).reshape(-1)
    tok = s["tok"].reshape(-1).clamp_min(0).long()
    flat = s["logits"].as_strided((B * N, V), (s["logits"].stride(1), 1))
    out = {"logp": torch.zeros(B * M, device=DEV), "entropy": torch.zeros(B * M, device=DEV)}
    if K:
        out["top_logp"] = torch.full((B * M, K), NEG_INF, device=DEV)
        out["top_tok"] = torch.full((B * M, K), -1, dtype=torch.int32, device=DEV)
    places = live.nonzero()[:, 0] if s["nodes"] is not None else torch.arange(B * M, device=DEV)
    for at in places.split(max(1, 100000000 // V)):
        x = flat[row[at]].float()
        y = x - x.max(-1, keepdim=True).values
        e = y.exp()
        z = e.sum(-1)
        lz = z.log()
        out["logp"][at] = y.gather(1, tok[at][:, None])[:, 0] - lz
        out["entropy"][at] = lz - torch.where(e > 0, e * y, torch.zeros_like(e)).sum(-1) / z
        if K:
            bits = (x + 0.0).view(torch.int32).long()  # order: the value, then the lower index
            bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
            key = bits * (1 << 32) + (0xFFFFFFFF - torch.arange(V, device=DEV))
            best = 0xFFFFFFFF - (key.topk(K, dim=-1).values & 0xFFFFFFFF)
            out["top_logp"][at] = y.gather(1, best) - lz[:, None]
            out["top_tok"][at] = best.int()
    return {k: v.reshape((B, M) + tuple(v.shape[1:])) for k, v in out.items()}


def _run_weights(s):
    case = s["case"]
    causal = s["nodes"] is not None
    if own:
        from ddtree_speculative_decode_b200 import lib
        if "ws" not in s:
            B, N, H, d = s["q"].shape
            n = lib.cache_weights_workspace_size(B, N, H, d, case["hi"], s["q"].dtype)
            s["ws"] = torch.zeros(max(n, 1), dtype=torch.uint8, device=s["q"].device)
        return lib.cache_weights(s["q"], s["lse"], s["kv"], s["score"], s["off"], s["len"], s["n"], case["scale"], case["hi"],
                                 nodes=s["nodes"], causal=causal, prev=s["prev"], decay=case["decay"], workspace=s["ws"])
    H = case["H"]
    lens, off, paths = s["len"].tolist(), s["off"].tolist(), _paths(case)
    for b, (n, o) in enumerate(zip(lens, off)):
        k = s["kv"][o:o + n].float()
        got = torch.zeros(n, device=DEV)
        nodes = s["nodes"][b, :paths[b]].long() if causal else torch.arange(case["N"], device=DEV)
        m = nodes.shape[0]
        step = max(1, 500000000 // (H * n))
        for i in range(0, m, step):
            at = nodes[i:i + step]
            y = case["scale"] * (s["q"][b, at].float().reshape(-1, case["d"]) @ k.T)
            p = (y - s["lse"][b, at].reshape(-1, 1)).exp()
            if causal:
                sees = n - m + 1 + i + torch.arange(at.shape[0], device=DEV).repeat_interleave(H)
                p = torch.where(torch.arange(n, device=DEV) < sees[:, None], p, torch.zeros_like(p))
            got += p.sum(0)
        s["score"][o:o + n] = case["decay"] * s["prev"][o:o + n] + got
    return s["score"]


def _run_evict(s):
    case = s["case"]
    outs = [s["dst_kv"], s["dst_score"], s["src"], s["new_len"]]
    if own:
        from ddtree_speculative_decode_b200 import lib
        if "ws" not in s:
            n = lib.cache_evict_workspace_size(case["B"], case["layers"], case["hi"])
            s["ws"] = torch.zeros(max(n, 1), dtype=torch.uint8, device=s["kv"].device)
        lib.cache_evict(s["kv"], s["score"], s["off"], s["len"], s["keep"], case["sink"], case["recent"], case["hi"],
                        n_layers=case["layers"], layer_stride_rows=s["rows"],
                        dst={"kv": s["dst_kv"], "score": s["dst_score"], "off": s["dst_off"], "layer_stride_rows": s["dst_rows"]},
                        out={"src": s["src"], "new_len": s["new_len"]}, workspace=s["ws"])
        return outs
    layers, d = case["layers"], case["d"]
    score, kv = s["score"].view(layers, -1), s["kv"].view(layers, -1, d)
    dst_score, dst_kv = s["dst_score"].view(layers, -1), s["dst_kv"].view(layers, -1, d)
    for b, (n, o, to) in enumerate(zip(s["lens"], s["offs"], s["dst_offs"])):  # ragged requests, all layers together
        m, x = min(n, case["keep"]), score[:, o:o + n]
        if m < n:
            order = x.clone()
            order[:, :case["sink"]] = float("inf")
            order[:, n - case["recent"]:] = float("inf")
            at = order.sort(dim=-1, descending=True, stable=True).indices[:, :m].sort(dim=-1).values
        else:
            at = torch.arange(n, device=DEV).expand(layers, n)
        s["src"][:, b, :m] = at.int()
        dst_kv[:, to:to + m] = kv[torch.arange(layers, device=DEV)[:, None], o + at]
        dst_score[:, to:to + m] = x.gather(1, at)
        s["new_len"][b] = m
    return outs


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------


def work(case):
    elt = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "logprobs":
        paths = _paths(case)
        rows = case["B"] * case["N"] if paths is None else sum(paths)
        return {"bytes": rows * (case["V"] * elt + 12 + 8 * case["K"]), "flops": 4 * rows * case["V"]}
    lens = _lens(case)
    if case["op"] == "weights":
        paths = _paths(case) or [case["N"]] * case["B"]
        d, H = case["d"], case["H"]
        return {"bytes": sum(n * (d * elt + 8) + m * H * (d * elt + 4) for n, m in zip(lens, paths)),
                "flops": sum(2 * n * m * H * d for n, m in zip(lens, paths))}
    kept = [min(n, case["keep"]) for n in lens]
    return {"bytes": case["layers"] * sum(4 * n + m * (2 * case["d"] * elt + 8) for n, m in zip(lens, kept)), "flops": 0}


# ---------------------------------------------------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        return _exact_logprobs(s)
    if case["op"] == "weights":
        return _exact_weights(s)
    return None  # nothing is computed: rows are chosen and copied


def _exact_logprobs(s):
    B, N, V = s["logits"].shape
    K, M = s["case"]["K"], s["tok"].shape[1]
    logp = torch.zeros((B, M), dtype=torch.float64, device=DEV)
    entropy = torch.zeros((B, M), dtype=torch.float64, device=DEV)
    top = torch.full((B, M, K), NEG_INF, dtype=torch.float64, device=DEV)
    for b in range(B):
        for j0 in range(0, M, 32):
            js = torch.arange(j0, min(M, j0 + 32), device=DEV)
            if s["nodes"] is not None:
                js = js[s["nodes"][b, js] >= 0]
            if not js.numel():
                continue
            rows = js if s["nodes"] is None else s["nodes"][b, js].long()
            lp = torch.log_softmax(s["logits"][b, rows].double(), -1)
            logp[b, js] = lp[torch.arange(js.numel(), device=DEV), s["tok"][b, js].long()]
            entropy[b, js] = -(lp.exp() * lp.clamp_min(-1e4)).sum(-1)
            if K:
                top[b, js] = lp.topk(K, -1).values
    out = {"logp": logp, "entropy": entropy}
    if K:
        out |= {"top_logp": top, "top_tok": None}
    return out


def _exact_weights(s):
    case = s["case"]
    score = torch.zeros_like(s["score"], dtype=torch.float64)
    for b in range(case["B"]):
        o, n = int(s["off"][b]), int(s["len"][b])
        keys = s["kv"][o:o + n].double()
        if s["nodes"] is None:
            rows = list(range(case["N"]))
        else:
            rows = [i for i in s["nodes"][b].tolist() if i >= 0]
        total = s["prev"][o:o + n].double() * case["decay"]
        for k, i in enumerate(rows):
            p = torch.exp(s["q"][b, i].double() @ keys.T * case["scale"] - s["lse"][b, i].double()[:, None])
            if s["nodes"] is not None:
                p[:, max(0, n - (len(rows) - 1 - k)):] = 0
            total += p.sum(0)
        score[o:o + n] = total
    return score
