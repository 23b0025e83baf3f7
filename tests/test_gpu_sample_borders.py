"""awq_sample at the border of min-p, where a weight and its nearest multiple of 2^-43 fall on different
sides of m: w_i >= m is asked of the weight itself, whichever way a row's tokens are found.

m is some 88 of the sums' units, 87.96 or 88.30 of them, and the packed logits' weights lie within a unit of it, so
some round across it, either way.  The random number is 1, so the token is the last one kept that has a weight: a token wrongly kept or
dropped is the answer itself.  The inputs have no weight within 2^-40 of m (relative), where 64 bits would not decide."""
import numpy as np
import pytest
import torch

import weight_only_quantization_gemm_amd as awq
from test_gpu_sample import choose

UNIT = 2.0 ** -43
B, PACKED = 64, 24
DEV = "cuda:0"


def rows(first, V, m, t, seed):
    """Logits [B][V]: `first` zeros, then -inf, and at the end packed ones whose weights at temperature t are
    within a unit of m.  The first of them in order is a zero."""
    g = np.random.default_rng(seed)
    l = np.full((B, V), -np.inf, np.float32)
    l[:, :first] = 0.0
    w = (m / UNIT + g.uniform(-0.9, 0.9, (B, PACKED))) * UNIT
    l[:, V - PACKED:] = np.float32(t) * np.log(w)
    exact = np.exp(l[:, V - PACKED:].astype(np.longdouble) / np.longdouble(np.float32(t)))
    assert np.abs(exact / np.longdouble(m) - 1).min() > 2.0 ** -40
    rounded = np.rint((exact / UNIT).astype(np.float64)) * UNIT
    crossing = (exact >= m) != (rounded >= m)
    assert crossing.any(1).sum() > B // 4  # rows with a token that rounds across m
    return l


@pytest.mark.gpu
@pytest.mark.parametrize("units", [87.96, 88.30])
@pytest.mark.parametrize("t", [1.0, 0.7, 1.9])
@pytest.mark.parametrize("first,V,top_k", [
    (1, 25, 0),            # one short list, cut by min-p
    (1, 60, 25), (20, 50, 44), (1, 5003, 25),  # a short list of the top-k
    (80, 5003, 104),       # a list to sort
    (80, 50021, 590), (80, 50021, 650), (400, 50021, 424),   # lists, or a histogram, by the kernel's size
    (80, 5003, 2000), (3000, 50021, 3024), (3000, 50021, 0),  # passes over the row
])
def test_min_p_is_asked_of_the_weight(first, V, top_k, t, units):
    m = float(np.float32(units * UNIT))
    logits = rows(first, V, m, t, seed=V + top_k)
    u = np.ones(B, np.float32)
    want = [choose(logits[b], t, top_k, 1.0, m, u[b]) for b in range(B)]
    dl, du = torch.from_numpy(logits).to(DEV), torch.from_numpy(u).to(DEV)
    every = lambda v, dtype: torch.full((B,), v, dtype=dtype, device=DEV)  # noqa: E731
    for k in (top_k, every(top_k, torch.int32)):
        for p in (m, every(m, torch.float32)):
            r = awq.awq_sample(dl, du, temperature=t, top_k=k, min_p=p)
            assert r["tokens"].tolist() == [token for token, _ in want]
            prob = np.array([prob for _, prob in want])
            # the quotient's rounding to fp32; a sum of at least 1 whose packed weights are within half a unit each
            assert np.all(np.abs(r["probs"].cpu().numpy() - prob) <= (2.0 ** -24 + PACKED * 2.0 ** -44) * prob)


@pytest.mark.gpu
@pytest.mark.parametrize("units", [87.96, 88.30])
@pytest.mark.parametrize("first,top_k", [(1, 25), (80, 104), (80, 650), (400, 424), (3000, 3024), (3000, 0)])
def test_min_p_in_the_longest_rows(first, top_k, units):
    """The same in rows of 2^20, whose chunks are too many for sums of each to be kept."""
    V, short, t = 1 << 20, first + PACKED, 1.0
    m = float(np.float32(units * UNIT))
    logits = rows(first, short, m, t, seed=first)
    want = [choose(logits[b], t, top_k, 1.0, m, np.float32(1)) for b in range(B)]
    dl = torch.full((B, V), -np.inf, device=DEV)
    dl[:, :first] = 0.0
    dl[:, V - PACKED:] = torch.from_numpy(logits[:, first:]).to(DEV)
    du = torch.ones(B, device=DEV)
    for k in (top_k, torch.full((B,), top_k, dtype=torch.int32, device=DEV)):
        tokens = awq.awq_sample(dl, du, temperature=t, top_k=k, min_p=m)["tokens"].tolist()
        assert tokens == [token if token < first else token + V - short for token, _ in want]


@pytest.mark.gpu
@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("value", [-3.25, float("inf")])
def test_the_largest_sum(value, half):
    """A row of 2^20 equal logits: each weighs 2^43 units, their sum is 2^63.  Of n that are kept the token is the whole
    part of u n, exactly, and its probability 1 / n to fp32's rounding."""
    V = 1 << 20
    u = np.array([0.0, 0.25, 0.5, 0.7, 1 - 2.0 ** -24, 1.0, 2.0], np.float32)
    logits = torch.full((len(u), V), value, dtype=torch.float16 if half else torch.float32, device=DEV)
    du = torch.from_numpy(u).to(DEV)
    for given, n in ((dict(), V), (dict(top_p=0.5), V // 2), (dict(top_k=V - 1), V - 1), (dict(top_k=700000, top_p=0.5), 350000),
                     (dict(min_p=1.0), V), (dict(top_p=0.75, min_p=0.5), 3 * V // 4)):
        r = awq.awq_sample(logits, du, **given)
        want = np.minimum(np.floor(u.astype(np.longdouble) * n), n - 1).astype(np.int64)  # 24 bits times 20
        assert r["tokens"].tolist() == want.tolist(), given
        assert np.all(np.abs(r["probs"].cpu().numpy() - 1 / n) <= 2.0 ** -24 / n)
