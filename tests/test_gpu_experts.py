"""Routing, plans, products grouped by expert and their weighted sum, against plain
implementations in 64 bits (numpy).

Tolerances.  A sum of n products in fp32 is off by at most n 2^-24 of the sum of their
magnitudes whatever its order (2^-23 allows a matrix core that truncates); rounding the result
to fp16 adds half a step, 2^-11 of it (2^-25 below the smallest normal number)."""
import numpy as np
import pytest
import torch

import weight_only_quantization_gemm_amd as awq
from layout import decode_codes, decode_codes3, decode_zeros, encode, encode3

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def note(text):
    print(text, flush=True)


# ---------------------------------------------------------------- route, plan
def route_ref(logits, k, renorm):
    """experts [T][k], weights (fp64), by the statement of awq_moe_route."""
    x = logits.astype(np.float64)
    T, E = x.shape
    experts, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        ok = [e for e in range(E) if x[t, e] > -np.inf]  # False for NaN
        order = sorted(ok, key=lambda e: (-x[t, e], e))[:k]
        if not order:
            continue
        p = {e: np.exp(x[t, e] - x[t, order[0]]) for e in ok}
        z = sum(p[e] for e in (order if renorm else ok))
        experts[t, :len(order)] = order
        weights[t, :len(order)] = [p[e] / z for e in order]
    return experts, weights


def plan_ref(experts, E):
    flat = experts.reshape(-1)
    kept = [p for e in range(E) for p in np.flatnonzero(flat == e)]
    dropped = np.flatnonzero((flat < 0) | (flat >= E))
    offsets = np.concatenate([[0], np.cumsum([np.sum(flat == e) for e in range(E)])]).astype(np.int32)
    pos = np.full(flat.size, -1, np.int32)
    pos[kept] = np.arange(len(kept))
    return offsets, np.concatenate([kept, dropped]).astype(np.int32), pos


def assert_plan(r, experts, E):
    offsets, rows, pos = plan_ref(experts, E)
    assert np.array_equal(host(r["offsets"]), offsets)
    assert np.array_equal(host(r["rows"]), rows)
    assert np.array_equal(host(r["pos"]), pos)


def assert_route(r, logits, k, renorm):
    experts, weights = route_ref(logits, k, renorm)
    assert np.array_equal(host(r["experts"]), experts)
    # exponent (difference of logits rounded: |d| 2^-24), exp (2 ulp, twice), a sum of E terms, a division
    x = logits.astype(np.float64)
    d = np.nan_to_num(np.where(np.isfinite(x), x, np.nan), nan=0.0)
    tol = (2 * np.ptp(d, axis=1)[:, None] + 8 + logits.shape[1]) * 2.0 ** -23
    w = host(r["weights"]).astype(np.float64)
    assert np.all(np.abs(w - weights) <= tol * weights + 2.0 ** -126)
    assert_plan(r, experts, logits.shape[1])


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (7, 64, 6), (32, 60, 8), (65, 65, 4), (200, 128, 8),
                                   (333, 256, 7), (40, 1000, 64), (2100, 16, 2), (1500, 1024, 8)])
@pytest.mark.parametrize("half", [True, False])
def test_route(T, E, k, half):
    note(f"route T={T} E={E} k={k} half={half}")
    g = np.random.default_rng(T + E + k)
    x = (g.standard_normal((T, E)) * 3).astype(np.float16 if half else np.float32)
    for renorm in (True, False):
        assert_route(awq.awq_moe_route(dev(x), k, renormalize=renorm), x, k, renorm)


@pytest.mark.parametrize("half", [True, False])
def test_route_ties_masks_and_lowest_values(half):
    """Equal logits go to the lower index; -inf and NaN are never chosen; the type's lowest
    value is an ordinary logit; a row with nothing left has no expert and no weight."""
    dt = np.float16 if half else np.float32
    low, E, k = np.finfo(dt).min, 70, 4
    x = np.zeros((9, E), dt)
    x[1, ::3] = 1.0                       # ties across lanes
    x[2] = -np.inf                        # nothing
    x[3] = -np.inf
    x[3, [69, 5]] = [2.0, 2.0]            # two left
    x[4] = low                            # all lowest: ordinary ties
    x[5] = low
    x[5, 33] = 1.0
    x[6] = np.nan
    x[6, 64] = -3.0
    x[7, 10:20] = np.nan
    x[7, 20:70] = -np.inf
    x[8] = -0.0
    x[8, 1::2] = 0.0                      # -0 and +0 are equal
    r = awq.awq_moe_route(dev(x), k)
    e = host(r["experts"])
    assert e[2].tolist() == [-1] * 4 and host(r["weights"])[2].tolist() == [0.0] * 4
    assert e[3].tolist() == [5, 69, -1, -1] and e[4].tolist() == [0, 1, 2, 3] and e[6].tolist() == [64, -1, -1, -1]
    for renorm in (True, False):
        assert_route(awq.awq_moe_route(dev(x), k, renormalize=renorm), x, k, renorm)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 3, 2), (130, 7, 8), (512, 8, 2), (1030, 33, 3), (40, 1024, 64),
                                   (9000, 64, 2)])
def test_plan(T, E, k):
    """Any choices: the same expert twice in a token, experts without a pair, dropped ids."""
    note(f"plan T={T} E={E} k={k}")
    g = np.random.default_rng(7 * T + E)
    experts = g.integers(-1, E + (1 if T > 3 else 0), size=(T, k)).astype(np.int32)
    if T > 3:
        experts[1] = E // 2
        experts[2, 0], experts[3, 0] = np.iinfo(np.int32).max, np.iinfo(np.int32).min
    assert_plan(awq.awq_moe_plan(dev(experts), E), experts, E)


def test_plan_of_nothing():
    experts = np.full((5, 2), -1, np.int32)
    assert_plan(awq.awq_moe_plan(dev(experts), 4), experts, 4)


# --------------------------------------------------------------------- product
def layer(E, N, K, bits, seed):
    """E random matrices: dequantised fp64 [E][N][K], magnitudes of (code + zero) scale, device arrays."""
    g = np.random.default_rng(seed)
    top = 16 if bits == 4 else 8
    q = g.integers(0, top, size=(E * N, K)).astype(np.uint8)
    z = g.integers(0, top, size=(E * N, K // 128)).astype(np.uint8)
    sc = (np.abs(g.standard_normal((E * N, K // 128))) * 0.01 + 1e-4).astype(np.float16)
    p, zb = (encode if bits == 4 else encode3)(q, z)
    dec = (decode_codes if bits == 4 else decode_codes3)(p, K)
    assert np.array_equal(dec, q) and np.array_equal(decode_zeros(zb, K // 128), z)
    w = (q.astype(np.float64) - np.repeat(z, 128, 1)) * np.repeat(sc.astype(np.float64), 128, 1)
    return w.reshape(E, N, K), dev(p.reshape(E, N, -1)), dev(sc.reshape(E, N, -1)), dev(zb.reshape(E, N, -1))


def inputs(M, K, seed):
    g = np.random.default_rng(seed)
    x = g.standard_normal((M, K))
    x[:, g.integers(0, K, size=max(1, K // 100))] *= 20
    return x.astype(np.float16)


def assert_rows(y, x, w, what, rounding=0.0):
    """y [n][N] against x [n][K] w^T; `rounding`: of x, relative."""
    ref = x.astype(np.float64) @ w.T
    mag = np.abs(x.astype(np.float64)) @ np.abs(w).T
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (w.shape[1] * 2.0 ** -23 + rounding) * mag
    y = y.astype(np.float64)
    with np.errstate(invalid="ignore"):
        near = np.abs(y - ref) <= tol
    # a sum of 65520 or more rounds to infinity in fp16
    near |= (y == np.copysign(np.inf, ref)) & (np.abs(ref) + tol >= 65520)
    assert near.all(), (what, int((~near).sum()), np.argwhere(~near)[:4].tolist())


def check_grouped(sizes, N, K, bits, seed, gather=None, scaled=False, extra=0):
    """sizes: rows of each expert; gather: top_k of a plan's rows; extra: rows after the last expert's."""
    E, R = len(sizes), int(sum(sizes)) + extra
    w, p, sc, z = layer(E, N, K, bits, seed)
    g = np.random.default_rng(seed + 1)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    kw = {}
    if gather:
        M = -(-R // gather) + 2
        x = inputs(M, K, seed + 2)
        rows = g.permutation(R).astype(np.int32)
        xr = x[rows // gather]
        kw = dict(rows=dev(rows), top_k=gather)
    else:
        x = xr = inputs(R, K, seed + 2)
    if scaled:
        s = np.exp(0.5 * g.standard_normal((E, K))).astype(np.float32)
        kw["s"] = dev(s)
    out = torch.full((R, N), 7.0, dtype=torch.float16, device=DEV)
    y = host(awq.awq_gemm_grouped(dev(x), p, sc, z, dev(offsets), out=out, **kw))
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            if scaled and (R > max(2 * E, 16) or "ring" not in awq.awq_gemm_grouped_kernel(R, E, N, K, bits)):
                xe = (xr[a:b].astype(np.float32) / s[e]).astype(np.float16)
                assert_rows(y[a:b], xe, w[e], f"expert {e}")
            elif scaled:  # two fp16 numbers: half a step of the second, 2^-11 of at most 2^-11 of x / s, and fp32's 2^-24
                assert_rows(y[a:b], xr[a:b].astype(np.float64) / s[e], w[e], f"expert {e}", 2.0 ** -22 + 2.0 ** -24)
            else:
                assert_rows(y[a:b], xr[a:b], w[e], f"expert {e}")
    assert np.all(y[offsets[-1]:] == 7.0), "rows behind the last expert were written"
    return y


SIZES = {
    "one row": [1],
    "one expert, one row of many": [0, 0, 1, 0],
    "none": [0, 0, 0],
    "few": [1, 0, 3, 2, 0, 0, 5, 1],
    "tile edges": [15, 16, 17, 0, 1, 31, 32, 33],
    "wide": [64, 0, 65, 63, 1],
    "large": [130, 2, 0, 257, 128],
    "many experts": [i % 4 for i in range(130)],
}


@pytest.mark.parametrize("bits", [4, 3])
@pytest.mark.parametrize("name", SIZES)
def test_grouped_sizes(name, bits):
    note(f"grouped sizes {name} bits={bits}")
    sizes = SIZES[name]
    N, K = (72, 256) if len(sizes) > 100 else (200, 384)
    check_grouped(sizes, N, K, bits, seed=len(name) + bits, extra=3)
    check_grouped(sizes, N, K, bits, seed=len(name) + bits + 50, gather=3, extra=3)


@pytest.mark.parametrize("bits", [4, 3])
@pytest.mark.parametrize("N,K", [(1, 128), (15, 128), (129, 640), (300, 1408), (64, 4096), (1000, 256), (17, 16640), (40, 131072)])
@pytest.mark.parametrize("rows", [1, 5, 40, 200])
def test_grouped_shapes(N, K, bits, rows):
    """Odd widths, one group, odd group counts and long rows, at few and many rows per expert."""
    note(f"grouped N={N} K={K} bits={bits} rows={rows}")
    check_grouped([rows, 0, 1 + rows // 3], N, K, bits, seed=N + K + bits + rows, gather=2)


@pytest.mark.parametrize("bits", [4, 3])
@pytest.mark.parametrize("rows", [1, 9, 70])
def test_grouped_scaled_input(bits, rows):
    note(f"grouped scaled bits={bits} rows={rows}")
    check_grouped([rows, 1, 0, 2 * rows], 136, 512, bits, seed=rows + bits, gather=2, scaled=True, extra=1)
    check_grouped([rows, 1, 0, 2 * rows], 136, 512, bits, seed=rows + bits, scaled=True)
    check_grouped([9, 8, 7, 0, 1] + [0] * 9, 136, 512, bits, seed=rows + bits, gather=2, scaled=True, extra=1)


@pytest.mark.parametrize("bits", [4, 3])
@pytest.mark.parametrize("rows", [1, 8])
def test_grouped_scaled_input_of_few_rows_is_not_rounded_to_fp16(bits, rows):
    """x / s enters with 22 bits: no larger error than the roundings of y itself (each at most half
    a step) and of fp32 sums leave, where x / s rounded to fp16 would miss by up to 2^-11 of each
    of a few large products.  An x / s above fp16's largest number is infinity."""
    N, K, E = 200, 512, 2
    w, p, sc, z = layer(E, N, K, bits, 41)
    x = inputs(2 * rows, K, 42)
    x[:, 5] *= 30
    s = np.exp(0.4 * np.random.default_rng(43).standard_normal((E, K))).astype(np.float32)
    off = dev(np.array([0, rows, 2 * rows], np.int32))
    assert "ring" in awq.awq_gemm_grouped_kernel(2 * rows, E, N, K, bits)
    y = host(awq.awq_gemm_grouped(dev(x), p, sc, z, off, s=dev(s)))
    for e in range(E):
        a = e * rows
        ref = (x[a:a + rows].astype(np.float64) / s[e]) @ w[e].T
        mag = np.abs(x[a:a + rows].astype(np.float64) / s[e]) @ np.abs(w[e]).T
        assert np.all(np.abs(y[a:a + rows] - ref) <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2.0 ** -20 * mag)
    x[0, 9], s[0, 9] = 60000, 0.25
    y = host(awq.awq_gemm_grouped(dev(x), p, sc, z, off, s=dev(s)))
    with np.errstate(invalid="ignore"):
        assert np.array_equal(y[0].astype(np.float64), np.inf * w[0, :, 9], equal_nan=True)


@pytest.mark.parametrize("bits", [4, 3])
@pytest.mark.parametrize("rows", [3, 150])
def test_grouped_scales_of_zero(bits, rows):
    """Groups whose scale is 0 add nothing, wherever they stand (the first group, the last, all of
    a row); scales of opposite extremes follow one another."""
    E, N, K = 2, 70, 768
    g = np.random.default_rng(rows + bits)
    w, p, sc, z = layer(E, N, K, bits, 9)
    s = host(sc).reshape(E * N, K // 128).copy()
    s[g.random(s.shape) < 0.3] = 0
    s[0], s[1, 0], s[2, -1] = 0, 0, 0
    s[3, ::2], s[3, 1::2] = 2.0 ** -14, 1000.0
    s[4, ::2], s[4, 1::2] = -0.01, 0.02
    q = (decode_codes if bits == 4 else decode_codes3)(host(p).reshape(E * N, -1), K).astype(np.float64)
    zz = decode_zeros(host(z).reshape(E * N, -1), K // 128)
    w = ((q - np.repeat(zz, 128, 1)) * np.repeat(s.astype(np.float64), 128, 1)).reshape(E, N, K)
    x = inputs(2 * rows, K, 10)
    x[:, :128] = np.abs(x[:, :128])
    y = host(awq.awq_gemm_grouped(dev(x), p, dev(s.reshape(E, N, -1)), z, dev(np.array([0, rows, 2 * rows], np.int32))))
    for e in range(E):
        assert_rows(y[e * rows:(e + 1) * rows], x[e * rows:(e + 1) * rows], w[e], f"expert {e}")
    assert np.all(y[:rows, 0] == 0)


@pytest.mark.parametrize("bits", [4, 3])
@pytest.mark.parametrize("rows", [1, 5, 80])
def test_grouped_infinite_input(bits, rows):
    """An infinity in x gives what the formula gives, infinities of the weight's sign and NaN where
    the weight is 0, in its own row; in the last of an odd number of groups, too."""
    N, K, at = 50, 640, 600
    w, p, sc, z = layer(2, N, K, bits, 31)
    x = inputs(2 * rows, K, 32)
    x[rows - 1, at] = np.inf
    y = host(awq.awq_gemm_grouped(dev(x), p, sc, z, dev(np.array([0, rows, 2 * rows], np.int32))))
    with np.errstate(invalid="ignore"):
        assert np.array_equal(y[rows - 1].astype(np.float64), np.inf * w[0, :, at], equal_nan=True)
    for e, lo, hi in ((0, 0, rows - 1), (1, rows, 2 * rows)):
        if lo < hi:
            assert_rows(y[lo:hi], x[lo:hi], w[e], f"expert {e}")


def test_grouped_matches_single_products_and_is_deterministic():
    """Each expert's rows are awq_gemm's product with its matrix, to rounding; two calls agree bit for bit."""
    sizes, N, K = [3, 0, 20, 1, 150], 256, 1024
    E = len(sizes)
    _, p, sc, z = layer(E, N, K, 4, 5)
    x = dev(inputs(sum(sizes), K, 6))
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    a = awq.awq_gemm_grouped(x, p, sc, z, dev(off))
    b = awq.awq_gemm_grouped(x, p, sc, z, dev(off))
    assert np.array_equal(host(a).view(np.uint16), host(b).view(np.uint16))
    for e in range(E):
        if sizes[e]:
            y = host(awq.awq_gemm(x[off[e]:off[e + 1]].contiguous(), p[e], sc[e], z[e])).astype(np.float64)
            d = host(a)[off[e]:off[e + 1]].astype(np.float64) - y
            assert np.linalg.norm(d) <= 2e-3 * np.linalg.norm(y)  # awq_gemm's own bar, twice


def test_grouped_bad_offsets_and_rows_stay_inside():
    """Offsets out of order or outside the batch and rows that lead outside x are kept inside by
    the kernel's clamps: nothing outside y's rows is written."""
    E, N, K, R = 3, 32, 128, 8
    _, p, sc, z = layer(E, N, K, 4, 1)
    x = dev(inputs(4, K, 2))
    big = np.iinfo(np.int32).max
    rows = dev(np.array([0, -5, big, 3, 100, 1, 2, 0], np.int32))
    for off in ([0, 100, 50, big], [-7, 3, 2, 8], [5, 4, 3, 2]):
        out = torch.full((R + 8, N), 7.0, dtype=torch.float16, device=DEV)
        awq.awq_gemm_grouped(x, p, sc, z, dev(np.array(off, np.int32)), rows=rows, out=out[:R])
        assert np.all(host(out)[R:] == 7.0)


# ----------------------------------------------------------------- combine, run
@pytest.mark.parametrize("T,k,N", [(1, 1, 8), (3, 2, 40), (50, 6, 2048), (257, 8, 1000), (5, 64, 128)])
def test_combine(T, k, N):
    note(f"combine T={T} k={k} N={N}")
    g = np.random.default_rng(T + k)
    y = g.standard_normal((T * k, N)).astype(np.float16)
    pos = g.permutation(T * k).astype(np.int32)
    pos[g.random(T * k) < 0.2] = -1
    if T > 2:
        pos[:k] = -1              # a token all of whose pairs were dropped
        pos[k] = T * k            # past the batch
    w = g.random((T, k)).astype(np.float32)
    ref, mag = np.zeros((T, N)), np.zeros((T, N))
    for p, r in enumerate(pos):
        if 0 <= r < T * k:
            ref[p // k] += w[p // k, p % k].astype(np.float64) * y[r]
            mag[p // k] += np.abs(w[p // k, p % k].astype(np.float64) * y[r])
    out = host(awq.awq_moe_combine(dev(y), dev(pos), dev(w))).astype(np.float64)
    assert np.all(np.abs(out - ref) <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + k * 2.0 ** -24 * mag)


@pytest.mark.parametrize("T", [1, 6, 90])
def test_expert_layer_together(T):
    """Router, gathered product, product of sorted rows, weighted sum: the layer of a token
    batch, eager and as a captured graph replayed on new inputs."""
    E, k, K, F = 8, 2, 256, 384
    w1, p1, s1, z1 = layer(E, F, K, 4, 11)
    w2, p2, s2, z2 = layer(E, K, F, 3, 12)
    g = np.random.default_rng(T)
    x, lg = torch.empty((T, K), dtype=torch.float16, device=DEV), torch.empty((T, E), device=DEV)

    def step():
        r = awq.awq_moe_route(lg, k)
        h = awq.awq_gemm_grouped(x, p1, s1, z1, r["offsets"], rows=r["rows"], top_k=k)
        y = awq.awq_gemm_grouped(h, p2, s2, z2, r["offsets"])
        return awq.awq_moe_combine(y, r["pos"], r["weights"]), r, h, y

    def fill():
        xs, l = inputs(T, K, int(g.integers(1 << 30))), g.standard_normal((T, E)).astype(np.float32)
        l[0] = -np.inf
        x.copy_(dev(xs))
        lg.copy_(dev(l))
        return xs, l

    xs, l = fill()
    out, r, h, y = step()
    assert_route(r, l, k, True)
    off, rows = host(r["offsets"]), host(r["rows"])
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a < b:
            assert_rows(host(h)[a:b], xs[rows[a:b] // k], w1[e], f"first product, expert {e}")
            assert_rows(host(y)[a:b], host(h)[a:b], w2[e], f"second product, expert {e}")
    assert np.all(host(out)[0] == 0.0)  # the token with no expert
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()[0]
    for _ in range(4):
        fill()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(captured).view(np.uint16), host(step()[0]).view(np.uint16))


def test_on_another_stream():
    _, p, sc, z = layer(2, 64, 128, 4, 3)
    x, off = dev(inputs(6, 128, 4)), dev(np.array([0, 2, 6], np.int32))
    a = host(awq.awq_gemm_grouped(x, p, sc, z, off))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = awq.awq_gemm_grouped(x, p, sc, z, off)
    side.synchronize()
    assert np.array_equal(a, host(b))


def test_refusals_of_the_binding():
    _, p, sc, z = layer(2, 64, 128, 4, 3)
    x, off = dev(inputs(6, 128, 4)), dev(np.array([0, 2, 6], np.int32))
    for kw in (dict(offsets=off[:2].contiguous()), dict(zeros=z[:1].contiguous()), dict(scales=sc[:, :1].contiguous()),
               dict(x=x[:, :64].contiguous()), dict(s=torch.ones(2, 64, device=DEV)), dict(x=x.t()),
               dict(out=torch.empty(5, 64, dtype=torch.float16, device=DEV))):
        with pytest.raises(ValueError):
            awq.awq_gemm_grouped(**{**dict(x=x, packed=p, scales=sc, zeros=z, offsets=off), **kw})
    with pytest.raises(TypeError):
        awq.awq_gemm_grouped(x.float(), p, sc, z, off)
    with pytest.raises(ValueError):
        awq.awq_moe_route(torch.zeros(2, 4, device=DEV), 5)
    with pytest.raises(TypeError):
        awq.awq_moe_route(torch.zeros(2, 4, device=DEV, dtype=torch.bfloat16), 2)
    with pytest.raises(awq.AwqError):
        awq.awq_moe_combine(torch.zeros(4, 12, device=DEV, dtype=torch.float16), torch.zeros(4, dtype=torch.int32, device=DEV),
                            torch.zeros(2, 2, device=DEV))
