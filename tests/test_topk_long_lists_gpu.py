"""Distillation from top logits with lists past one pass of the row kernels
(128 entries), up to the longest (1,024)."""
import pytest
import torch

from test_topk_gpu import make, run_all

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [3, 40])
@pytest.mark.parametrize("pad", [False, True])
@pytest.mark.parametrize("K,V", [(129, 132), (129, 5003), (257, 260), (257, 4096), (1023, 1030), (1023, 6001),
                                 (1024, 1024), (1024, 3001)])
def test_long_lists(N, K, V, pad):
    c = make(N, 64, V, K, seed=41, pad=pad, whole=True, weights=pad)
    for tail in (False, True):
        run_all(c, tail=tail)


@pytest.mark.parametrize("N", [2, 300])
@pytest.mark.parametrize("K", [130, 513, 1024])
def test_an_id_listed_twice_on_both_sides_of_a_pass(N, K):
    """Equal ids at the sorted places 127 and 128, and at 63, 64 and 65."""
    c = make(N, 64, 2500, K, seed=42, whole=True)
    order = c["ids"].argsort(1)
    for a, b in ((127, 128), (64, 63), (64, 65)):
        c["ids"].scatter_(1, order[:, b:b + 1], c["ids"].gather(1, order[:, a:a + 1]))
    assert bool((c["ids"].sort(1).values[:, 127] == c["ids"].sort(1).values[:, 128]).all())
    c["lse_t"] += 0.5
    run_all(c, tail=True)
    c["lse_t"] = None
    run_all(c)


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("logits", [torch.bfloat16, torch.float16])
def test_long_lists_of_every_type(ids, logits):
    run_all(make(150, 128, 3000, 600, seed=43, ids_dtype=ids, logits_dtype=logits, mask=True, pad=True))
