"""The draw at an infinite temperature, where fewer tokens are left than the K that are
drawn from: those left weigh the same, the rest nothing.  The expected tokens are written
out by hand: of n tokens left, u draws number floor(n u)."""
import numpy as np
import pytest

from oracle import rules

INF = float("inf")
U = [0.0, 0.125, 0.25, 0.5, 0.625, 0.75, 0.9375]  # no border of 3 or 5 tokens among them
LEFT = {1: [7], 3: [40, 7, 59], 5: [40, 7, 59, 0, 22]}  # in the order of their logits


@pytest.mark.parametrize("n", LEFT)
def test_oracle(n):
    values = np.concatenate([3.0 - np.arange(n), np.full(16 - n, -INF)])
    ids = np.concatenate([LEFT[n], 100 + np.arange(16 - n)])
    for u in U:
        assert rules.draw(values, ids, u, INF) == LEFT[n][int(n * u)]


def test_oracle_without_anything_banned():
    assert [rules.draw([2.0, 1.0, 1.0, -5.0], [4, 1, 3, 0], u, INF) for u in (0.0, 0.3, 0.6, 0.9)] == [4, 1, 3, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("way", ["logits", "mask", "biases"])
@pytest.mark.parametrize("n", LEFT)
def test_kernel(n, way):
    import torch
    import packed_quantized_lm_amd as pq
    V, M = 60, len(U)
    y = np.full((M, V), -9.0, dtype=np.float32)
    y[:, LEFT[n]] = 3.0 - np.arange(n)
    banned = np.setdiff1d(np.arange(V), LEFT[n]).astype(np.int32)
    kw = {}
    if way == "logits":
        y[:, banned] = -INF
    elif way == "mask":
        kw["mask"] = torch.from_numpy(rules.bits(np.tile(np.isin(np.arange(V), LEFT[n]), (M, 1)))).cuda()
    else:
        kw["bias_ids"] = torch.from_numpy(banned).cuda()
        kw["bias_values"] = torch.full((len(banned),), -INF, device="cuda")
    for K in (n, n + 1, 16):
        _, ids, drawn = pq.sample_logits(torch.from_numpy(y).cuda(), K, u=torch.tensor(U, device="cuda"),
                                         temperature=torch.full((M,), INF, device="cuda"), **kw)
        assert ids[:, :n].tolist() == [LEFT[n]] * M
        assert drawn.tolist() == [LEFT[n][int(n * u)] for u in U], K
