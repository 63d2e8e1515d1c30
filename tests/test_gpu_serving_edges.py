"""Rare paths of the token-score and cache-budget calls: what ordinary inputs
seldom reach, each against a plain computation."""
import numpy as np
import pytest
import torch

from ddtree_speculative_decode_b200 import lib
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
