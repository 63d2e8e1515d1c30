"""Token scores and the cache budget as they are used together.

On the tiny MLA decoder, the library's loop (attention -> accept -> token
log-probs, cache weights -> eviction, on every layer) against a float64 loop
on the CPU around the oracle's forward: the same tokens, scores and remaining
latent rows. And at MLA serving size, one step of the calls on bf16 inputs
against plain 64-bit arithmetic. This file sorts after the other GPU tests."""
import numpy as np
import pytest
import torch

import oracle
from oracle import spec_loop
from ddtree_speculative_decode_b200 import lib, spec_engine, synth
from ddt_testutil import golden_drafter, step_to_device, t_from

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PROMPT = [3, 14, 15, 92, 65]


class Plain:
    """The loop in float64: oracle forward, explicit weights and evictions."""

    def __init__(self, w, monkeypatch, budget, sink, recent, decay, capacity=128):
        self.w, self.budget, self.sink, self.recent, self.decay = w, budget, sink, recent, decay
        self.cache = spec_loop.LatentCache(w, capacity)
        self.score = np.zeros((self.cache.n_layers, capacity))
        self.evicted = 0
        self.gap = np.inf  # smallest distance between a kept and a dropped score, relative to them
        self.seen = []
        plain_attn = oracle.verify_attn

        def attn(q, pool, off, L, mask, n, H, dl, dr, scale, dtype):
            out, lse = plain_attn(q, pool, off, L, mask, n, H, dl, dr, scale, dtype)
            self.seen.append((q[0], lse[0]))
            return out, lse

        monkeypatch.setattr(spec_loop, "verify_attn", attn)

    def rows(self, toks, pos, mask):
        self.seen = []
        return spec_loop.forward_rows(self.w, self.cache, toks, np.asarray(pos) + self.evicted, mask)

    def hold(self, path):
        c = self.cache
        L, m = c.length, len(path)
        for li, (q, lse) in enumerate(self.seen):
            s = self.score[li]
            s[L - m:L] = 0.0
            s[:L] *= self.decay
            keys = c.layer(li)[:L]
            for k, i in enumerate(path):
                p = np.exp(self.w["scale"] * (q[i] @ keys.T) - lse[i][:, None])
                p[:, L - m + 1 + k:] = 0.0
                s[:L] += p.sum(0)
        if L <= self.budget:
            return
        for li in range(c.n_layers):
            s, pool = self.score[li], c.layer(li)
            middle = np.arange(self.sink, L - self.recent)
            order = middle[np.argsort(-s[middle], kind="stable")]
            n = self.budget - self.sink - self.recent
            a, b = s[order[n - 1]], s[order[n]]
            self.gap = min(self.gap, (a - b) / a)
            kept = np.sort(np.concatenate([np.arange(self.sink), order[:n], np.arange(L - self.recent, L)]))
            s[:self.budget] = s[kept].copy()
            pool[:self.budget] = pool[kept].copy()
        self.evicted += L - self.budget
        c.length = self.budget

    def one(self, tok):
        lg = self.rows([tok], [self.cache.length], np.ones((1, 1), np.uint32))
        self.cache.length += 1
        self.hold([0])
        return int(lg[0].argmax()), lg[0]

    def ddtree(self, T, drafter, block, K):
        nxt = None
        for t in PROMPT:
            nxt, _ = self.one(t)
        committed, scores, c = [nxt], [], self.cache
        while len(committed) < T:
            lp, tk = drafter(committed, block - 1, K)
            L = c.length
            tree = oracle.build_tree(lp[None], tk[None], np.array([committed[-1]]), np.array([L]), block)
            n = int(tree["n_nodes"][0])
            logits = np.zeros((1, block, self.w["V"]))
            logits[0, :n] = self.rows(tree["node_tok"][0, :n], tree["pos"][0, :n], tree["mask"][0, :n])
            r = oracle.accept_compact(logits, "f32", tree["node_tok"], tree["parent"], tree["n_nodes"], c.kv, np.array([0]),
                                      np.array([L], np.int32), np.array([c.stride], np.int32), n_layers=c.n_layers,
                                      layer_stride_rows=c.stride)
            a = int(r["acc_len"][0])
            path = [int(x) for x in r["acc_nodes"][0, :a + 1]]
            toks = [int(x) for x in r["out_tok"][0, :a + 1]]
            committed += toks
            c.length = L + a + 1
            for i, t in zip(path, toks):
                x = logits[0, i] - logits[0, i].max()
                lpx = x - np.log(np.exp(x).sum())
                order = np.argsort(-logits[0, i], kind="stable")[:4]
                scores.append((lpx[t], -(np.exp(lpx) * lpx).sum(), order.tolist(), lpx[order]))
            self.hold(path)
        return committed, scores


@pytest.fixture(scope="module")
def weights():
    return synth.tiny_mla_weights()


@pytest.mark.parametrize("budget,sink,recent,decay,p_hit", [(16, 2, 6, 1.0, 1.0), (24, 4, 8, 0.9, 0.6), (12, 0, 0, 0.8, 0.6),
                                                            (100, 0, 0, 1.0, 0.6)])
def test_generation_within_a_budget(weights, monkeypatch, budget, sink, recent, decay, p_hit):
    golden, _ = spec_loop.ar_generate(weights, PROMPT, 60)
    plain = Plain(weights, monkeypatch, budget, sink, recent, decay)
    want, scores = plain.ddtree(40, golden_drafter(golden, weights["V"], p_hit, 3), 8, 3)
    # what is compared must not hang on a float32 rounding: the chosen scores
    # stay further apart than float32 sums of a few hundred terms can move
    assert plain.gap > 2e-5
    eng = spec_engine.TinyMLAEngine(weights, 128, cache_budget=budget, sink=sink, recent=recent, decay=decay)
    got, steps, gs = eng.ddtree_generate(PROMPT, 40, golden_drafter(golden, weights["V"], p_hit, 3), 8, 3, logprobs=4)
    assert got == want
    assert eng.length == plain.cache.length <= budget and eng.evicted == plain.evicted
    assert (eng.evicted > 0) == (budget < 45)
    for li in range(eng.n_layers):
        np.testing.assert_allclose(eng.layer(li)[:eng.length].cpu().numpy(), plain.cache.layer(li)[:eng.length], rtol=1e-4,
                                   atol=1e-5)
        np.testing.assert_allclose(eng.score[li * 128:li * 128 + eng.length].cpu().numpy(), plain.score[li][:eng.length],
                                   rtol=1e-4, atol=1e-5)
    assert len(gs) == len(scores) == len(got) - 1
    for (a, b, c, d), (e, f, g, h) in zip(gs, scores):
        assert abs(a - e) < 1e-4 and abs(b - f) < 1e-4 and c == g and np.abs(np.array(d) - h).max() < 1e-4


def test_a_budget_that_holds_everything_changes_nothing(weights):
    eng = spec_engine.TinyMLAEngine(weights, 128)
    golden = eng.ar_generate(PROMPT, 40)
    ref = spec_engine.TinyMLAEngine(weights, 128)
    want = ref.ddtree_generate(PROMPT, 30, golden_drafter(golden, weights["V"], 0.6, 1), 8, 3)
    eng = spec_engine.TinyMLAEngine(weights, 128, cache_budget=128)
    assert eng.ddtree_generate(PROMPT, 30, golden_drafter(golden, weights["V"], 0.6, 1), 8, 3) == want
    assert torch.equal(eng.kv, ref.kv) and eng.evicted == 0


def test_engine_refuses_budgets_that_cannot_hold(weights):
    for kw in (dict(cache_budget=0), dict(cache_budget=129), dict(cache_budget=10, sink=4, recent=7)):
        with pytest.raises(ValueError):
            spec_engine.TinyMLAEngine(weights, 128, **kw)


def test_one_serving_step():
    """build -> attention -> accept -> token log-probs and cache weights -> eviction on two layers, bf16 MLA rows."""
    s = synth.custom("budget-bf16", B=3, D=6, K=4, N=24, H=64, d_l=512, d_r=64, V=3001, L=(700, 90, 333), dtype="bf16",
                     kv_scale=1.0, scale=1.0 / np.sqrt(192.0), seed=21)
    x = synth.make_step(s)
    d = step_to_device(x, DEV)
    rows, B = x.kv.shape[0], s.B
    tree = lib.build_tree(d["logp"], d["tok"], d["root_tok"], d["cache_len"], s.N)
    g = torch.Generator(device=DEV).manual_seed(3)
    kv = torch.stack([d["kv"], torch.randn(rows, 576, device=DEV, generator=g).bfloat16()]).reshape(-1, 576).contiguous()
    score = torch.rand(2 * rows, device=DEV, generator=g)
    qs = [d["q"], torch.randn(d["q"].shape, device=DEV, generator=g).bfloat16()]
    lses = [lib.verify_attn(q, kv[la * rows:(la + 1) * rows], d["cache_off"], d["cache_len"], tree["mask"], tree["n_nodes"],
                            512, 64, s.scale, 700)[1] for la, q in enumerate(qs)]
    host = {k: tree[k].cpu().numpy() for k in ("parent", "node_tok", "n_nodes")}
    logits = t_from(synth.target_logits(s, host["parent"], host["node_tok"], host["n_nodes"]), DEV, True)
    cl = d["cache_len"].clone()
    acc = lib.accept_compact(logits, tree["node_tok"], tree["parent"], tree["n_nodes"], kv, d["cache_off"], cl,
                             d["cache_cap"], n_layers=2, layer_stride_rows=rows)
    lp = lib.token_logprobs(logits, acc["out_tok"], nodes=acc["acc_nodes"], K=3)
    before, base, lens = kv.clone(), score.clone(), cl.tolist()
    off = d["cache_off"].tolist()
    path = [[i for i in r if i >= 0] for r in acc["acc_nodes"].tolist()]
    assert [n - m for n, m in zip(lens, map(len, path))] == [700, 90, 333] and max(map(len, path)) > 2
    for la, (q, lse) in enumerate(zip(qs, lses)):
        sc = score[la * rows:(la + 1) * rows]
        lib.cache_weights(q, lse, kv[la * rows:(la + 1) * rows], sc, d["cache_off"], cl, tree["n_nodes"], s.scale, 710,
                          nodes=acc["acc_nodes"], causal=True, prev=sc, decay=0.95)
    keep = torch.tensor([400, 200, 200], dtype=torch.int32, device=DEV)
    weighed = score.clone()
    out = lib.cache_evict(kv, score, d["cache_off"], cl, keep, 4, 32, 710, n_layers=2, layer_stride_rows=rows)
    torch.cuda.synchronize()
    for b in range(B):
        for j, i in enumerate(path[b]):
            lpx = torch.log_softmax(logits[b, i].double(), -1)
            t = int(acc["out_tok"][b, j])
            assert abs(float(lp["logp"][b, j]) - float(lpx[t])) < 2e-5
            assert int(lp["top_tok"][b, j, 0]) == t == int(acc["am"][b, i])  # greedy: the most likely token
            assert abs(float(lp["entropy"][b, j]) + float((lpx.exp() * lpx).sum())) < 2e-5
        assert bool((lp["logp"][b, len(path[b]):] == 0).all())
        for la, (q, lse) in enumerate(zip(qs, lses)):
            a, n, m = la * rows + off[b], lens[b], len(path[b])
            keys = before[a:a + n].double()
            w = base[a:a + n].double() * 0.95
            for k, i in enumerate(path[b]):
                p = torch.exp(s.scale * (q[b, i].double() @ keys.T) - lse[b, i].double()[:, None])
                p[:, n - m + 1 + k:] = 0
                # a verify row's weights over what it sees add up to one (lse is bf16 attention's float32 one)
                assert float((p.sum(-1) - 1).abs().max()) < 2e-3
                w += p.sum(0)
            got = weighed[a:a + n].double()
            assert float(((got - w).abs() / w).max()) < 1e-4
            kept = min(n, int(keep[b]))
            idx = out["src"][la, b, :kept].long()
            assert torch.equal(kv[a:a + kept], before[a + idx]) and torch.equal(score[a:a + kept], weighed[a + idx])
            if n > kept:
                order = weighed[a:a + n].clone()
                order[:4] = np.inf
                order[n - 32:] = np.inf
                want = torch.sort(order, descending=True, stable=True).indices[:kept].sort().values
                assert torch.equal(idx, want)
    assert cl.tolist() == [400, len(path[1]) + 90, 200]
    # the next step reads the shortened caches
    tree2 = lib.build_tree(d["logp"], d["tok"], acc["bonus"], cl, s.N)
    o, l = lib.verify_attn(qs[0], kv[:rows], d["cache_off"], cl, tree2["mask"], tree2["n_nodes"], 512, 64, s.scale, 710)
    ref, rl = oracle.verify_attn(x.q, kv[:rows].view(torch.int16).cpu().numpy().view(np.uint16), x.cache_off,
                                 cl.cpu().numpy(), tree2["mask"].cpu().numpy().view(np.uint32),
                                 tree2["n_nodes"].cpu().numpy(), 64, 512, 64, s.scale, "bf16")
    assert float(np.abs(o.float().cpu().numpy() - ref).max()) <= 2e-2 * np.abs(ref).max()
