"""awq_sample against its definition, row by row on the host with weights in extended precision.

Tokens are whole numbers and have to be equal: the kernel's sums are exact multiples of 2^-43, the
oracle's within 2^-60, so they can only differ where a random number falls within about 2^-40 of a
border, which the seeds here do not.  A probability is a quotient rounded to fp32 (2^-24) of weights
in multiples of 2^-43; the oracle's own is exact beside that."""
import numpy as np
import pytest
import torch

import weight_only_quantization_gemm_amd as awq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def choose(l, t, k, p, m, u):
    """(token, probability) of one row."""
    l = l.astype(np.float32)
    live = np.flatnonzero(l > -np.inf)  # NaN is not
    if live.size == 0:
        return -1, 0.0
    order = live[np.lexsort((live, -l[live].astype(np.float64)))]
    top = l[order[0]]
    if not t > 0:
        return int(order[0]), 1.0
    v = l[order].astype(np.longdouble)
    with np.errstate(all="ignore"):
        w = np.where(l[order] == top, np.longdouble(1), np.exp((v - np.longdouble(top)) / np.longdouble(np.float32(t))))
    w = np.where(w >= 2.0 ** -44, w, np.longdouble(0))  # false for a NaN
    if 1 <= k < l.size:
        order, w = order[:k], w[:k]
    if p < 1:
        before = np.cumsum(w) - w
        keep = before < np.longdouble(np.float32(p)) * w.sum()
        keep[0] = True
        order, w = order[keep], w[keep]
    if m > 0:
        keep = w >= np.longdouble(np.float32(m))
        keep[0] = True
        order, w = order[keep], w[keep]
    back = np.argsort(order)
    order, w = order[back], w[back]
    upto = np.cumsum(w)
    u = np.float32(u)
    target = (np.longdouble(u) if u > 0 else np.longdouble(0)) * upto[-1]
    over = np.flatnonzero(upto > target)
    at = int(over[0]) if over.size else int(np.flatnonzero(w > 0)[-1])
    return int(order[at]), float(w[at] / upto[-1])


def check(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, rows=None, dev_logits=None):
    B = len(logits)
    dl = torch.from_numpy(logits).to(DEV) if dev_logits is None else dev_logits
    settings = dict(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    given = {n: (torch.from_numpy(v).to(DEV) if isinstance(v, np.ndarray) else v) for n, v in settings.items()}
    r = awq.awq_sample(dl, torch.from_numpy(u.astype(np.float32)).to(DEV), **given)
    tokens, probs = r["tokens"].cpu().numpy(), r["probs"].cpu().numpy()
    at = lambda v, b: v[b] if isinstance(v, np.ndarray) else v  # noqa: E731
    for b in range(B) if rows is None else rows:
        token, prob = choose(logits[b], *(at(settings[n], b) for n in ("temperature", "top_k", "top_p", "min_p")), u[b])
        assert tokens[b] == token, (b, tokens[b], token)
        assert abs(probs[b] - prob) <= (2.0 ** -24 + 2.0 ** -40) * prob + 2.0 ** -42, (b, probs[b], prob)
    return r


def logits_of(B, V, seed, half, spread=2.0):
    g = np.random.default_rng(seed)
    l = spread * g.standard_normal((B, V)) + np.where(g.random((B, V)) < 20 / V, 5.0, 0.0)
    return l.astype(np.float16 if half else np.float32), g.random(B).astype(np.float32)


FILTERS = [dict(), dict(top_k=1), dict(top_k=5), dict(top_k=50, temperature=0.7), dict(top_k=700), dict(top_p=0.9),
           dict(top_p=0.5, temperature=1.5), dict(top_p=0.999), dict(min_p=0.05), dict(top_k=40, top_p=0.95, min_p=0.02),
           dict(top_k=300, top_p=0.3), dict(temperature=0.0), dict(temperature=8.0, top_p=0.7), dict(top_p=1e-6),
           dict(temperature=0.05, top_k=20, top_p=0.9), dict(top_k=3000, top_p=0.99, temperature=3.0)]


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("f", FILTERS, ids=str)
def test_filters(f, half):
    for V in (1, 2, 7, 64, 1000, 4099, 50021):
        check(*logits_of(12, V, seed=V, half=half), **f)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("B,V", [(1, 32000), (3, 131072), (2, 152001), (1, 1 << 20), (300, 333), (700, 1024), (65, 9000)])
def test_sizes_with_settings_for_each_row(B, V, half):
    g = np.random.default_rng(B)
    logits, u = logits_of(B, V, seed=V + B, half=half)
    rows = None if B * V < 4e6 else range(0, B, max(1, B // 40))
    check(logits, u, temperature=g.choice([0.0, 0.5, 1.0, 2.0], B).astype(np.float32),
          top_k=g.choice([0, -3, 1, 10, 64, V, V + 5], B).astype(np.int32),
          top_p=g.choice([1.0, 0.95, 0.6, 2.0], B).astype(np.float32),
          min_p=g.choice([0.0, 0.1, 0.01, -1.0], B).astype(np.float32), rows=rows)
    check(logits, u, top_k=20, top_p=0.9, rows=rows)
    check(logits, u, top_p=0.97, rows=rows)
    check(logits, u, rows=rows)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("V", [5, 1000, 40000])
def test_equal_logits(V, half):
    """Ties go to the lowest index, also at the border of top-k and top-p, exactly."""
    logits = np.full((9, V), -3.25, np.float16 if half else np.float32)
    u = np.array([0.0, 0.5, 0.25, 0.999999, 0.125, 0.75, 0.3, 0.6, 0.9], np.float32)
    for f in (dict(), dict(top_k=3), dict(top_p=0.5), dict(top_k=V // 2, top_p=0.5), dict(min_p=1.0), dict(top_p=0.0)):
        check(logits, u, **f)
    # a few values, each many times
    g = np.random.default_rng(V)
    logits = g.choice([-2.0, 0.0, 0.5, 1.0, -np.inf], (9, V)).astype(logits.dtype)
    for f in (dict(), dict(top_k=V // 3 + 1), dict(top_p=0.7), dict(top_k=V // 2 + 1, top_p=0.81), dict(min_p=0.6)):
        check(logits, u, **f)


@pytest.mark.parametrize("half", [True, False])
def test_masked_infinite_and_nan_logits(half):
    V = 3001
    logits, u = logits_of(12, V, seed=3, half=half)
    logits[0] = -np.inf
    logits[1] = np.nan
    logits[2, 5:] = -np.inf
    logits[3, :-1] = -np.inf
    logits[4, ::2] = np.nan
    logits[5, [100, 2000, 2500]] = np.inf
    logits[6] = np.finfo(logits.dtype).min
    logits[7, 10:] = np.finfo(logits.dtype).min
    logits[8] = np.inf
    logits[9] = 0.0
    logits[9, ::3] = -0.0
    for f in (dict(), dict(top_k=2), dict(top_p=0.9), dict(top_k=10, top_p=0.5, min_p=0.1), dict(temperature=0.0),
              dict(temperature=float("inf")), dict(temperature=1e-30), dict(temperature=1e30, top_k=7)):
        r = check(logits, u, **f)
        assert r["tokens"][:2].tolist() == [-1, -1] and r["probs"][:2].tolist() == [0.0, 0.0]


def test_random_numbers_outside_the_range():
    logits, _ = logits_of(6, 500, seed=1, half=False)
    logits[:, 400:] = -1000.0  # of no weight: the last token with one is below 400
    u = np.array([0.0, -1.0, np.nan, 1.0, 7.0, np.inf], np.float32)
    for f in (dict(), dict(top_k=30), dict(top_p=0.8)):
        r = check(logits, u, **f)
        assert r["tokens"].max().item() < 400


def test_settings_that_are_no_numbers_are_off():
    logits, u = logits_of(4, 700, seed=2, half=True)
    nan = np.full(4, np.nan, np.float32)
    a = check(logits, u, top_p=nan, min_p=nan)
    assert torch.equal(a["tokens"], check(logits, u)["tokens"])
    check(logits, u, temperature=nan)


@pytest.mark.parametrize("V", [40, 700, 20011])
def test_top_p_that_is_no_number_beside_other_settings(V):
    logits, u = logits_of(6, V, seed=V, half=True)
    nan = np.full(6, np.nan, np.float32)
    for f in (dict(top_k=5), dict(top_k=90), dict(top_k=650), dict(min_p=0.02), dict(top_k=30, min_p=0.1)):
        check(logits, u, top_p=nan, **f)


@pytest.mark.parametrize("half", [True, False])
def test_signalling_nan_is_never_chosen(half):
    logits, u = logits_of(6, 5003, seed=8, half=half)
    bits = logits.view(np.uint16 if half else np.uint32)
    g = np.random.default_rng(4)
    for v in (0x7C01, 0xFC01, 0x7DFF, 0x7E00) if half else (0x7F800001, 0xFF800001, 0x7FBFFFFF, 0x7FC00000):
        bits[:, g.choice(5003, 500)] = v
    for f in (dict(), dict(top_k=20), dict(top_p=0.8), dict(temperature=0.0)):
        check(logits, u, **f)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("stride", [1003, 1008, 1500, 1001])
def test_strided_rows(half, stride):
    logits, u = logits_of(7, 1001, seed=6, half=half)
    wide = torch.full((7, stride), 50.0, dtype=torch.float16 if half else torch.float32, device=DEV)
    wide[:, :1001] = torch.from_numpy(logits).to(DEV)
    for f in (dict(), dict(top_k=30, top_p=0.9), dict(top_p=0.6)):
        check(logits, u, dev_logits=wide[:, :1001], **f)


def test_distribution():
    """Over evenly spaced random numbers each token comes up in proportion to its weight, to one
    step of the spacing."""
    g = np.random.default_rng(5)
    n = 4096
    row = g.standard_normal(30).astype(np.float32)
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    r = awq.awq_sample(torch.from_numpy(np.tile(row, (n, 1))).to(DEV), torch.from_numpy(u).to(DEV), temperature=0.9)
    count = np.bincount(r["tokens"].cpu().numpy(), minlength=30)
    w = np.exp(row.astype(np.float64) / np.float64(np.float32(0.9)))
    assert np.all(np.abs(count - n * w / w.sum()) <= 1.01)


def test_repeats_stream_and_graph():
    logits, u = logits_of(40, 20011, seed=9, half=True)
    dl, du = torch.from_numpy(logits).to(DEV), torch.from_numpy(u).to(DEV)
    call = lambda: awq.awq_sample(dl, du, temperature=0.9, top_k=100, top_p=0.9)  # noqa: E731
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    assert torch.equal(got["tokens"], want["tokens"]) and torch.equal(got["probs"], want["probs"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for i in range(3):
        du.copy_((du + 0.3) % 1.0)
        dl.copy_(dl.roll(17, dims=1))
        want = call()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got["tokens"], want["tokens"]) and torch.equal(got["probs"], want["probs"])


def test_refusals():
    l, u = torch.zeros(3, 50, device=DEV), torch.zeros(3, device=DEV)
    for bad in (lambda: awq.awq_sample(l, u[:2]), lambda: awq.awq_sample(l, u, top_k=torch.zeros(2, dtype=torch.int32, device=DEV)),
                lambda: awq.awq_sample(l.t(), torch.zeros(50, device=DEV)), lambda: awq.awq_sample(l, u.cpu()),
                lambda: awq.awq_sample(l, u, top_k=2 ** 32 + 1), lambda: awq.awq_sample(l, u, top_k=-2 ** 31 - 1),
                lambda: awq.awq_sample(l, u, temperature=float("nan")), lambda: awq.awq_sample(l[:, :0], u)):
        with pytest.raises((ValueError, awq.AwqError)):
            bad()
    for bad in (lambda: awq.awq_sample(l, u, top_k=torch.zeros(3, device=DEV)), lambda: awq.awq_sample(l, u.double()),
                lambda: awq.awq_sample(l, u, top_p=torch.ones(3, dtype=torch.float16, device=DEV))):
        with pytest.raises(TypeError):
            bad()
