"""The grouped product's large tiles by value: every kernel that the dispatch can choose, at sizes
where its row blocks are full, partly full and empty; and routes of more than 900 experts in one
launch."""
import numpy as np
import pytest

import weight_only_quantization_gemm_amd as awq
from layout import decode_codes, decode_codes3, decode_zeros
from test_gpu_experts import DEV, assert_plan, assert_route, assert_rows, check_grouped, dev, host, inputs, layer, note

# rows of each expert, N, K, and the kernel (of each code width) that serves them
TILES = [
    ([1, 0, 2, 0, 0, 0, 0], 40, 384, "grouped_ring_kernel<{},2,2>"),
    ([3, 9, 0, 8], 40, 384, "grouped_ring_kernel<{},4,2>"),
    ([70, 31, 0, 63, 97, 64], 300, 384, "grouped_pipe_kernel<{},2,1,3>"),
    ([70, 31, 0, 63, 97, 64], 40, 24576, "grouped_pipe_kernel<{},2,1,2>"),
    ([900, 1, 300, 420], 300, 384, "grouped_pipe_kernel<{},4,2,3>"),
    ([257, 33, 800, 129, 710], 260, 256, "grouped_pipe_kernel<{},4,2,3>"),
    ([0, 1600, 32, 64, 96, 128, 160, 192, 224, 1600], 70, 128, "grouped_pipe_kernel<{},4,2,3>"),
    ([401, 290, 470], 40, 11008, "grouped_pipe_kernel<{},4,2,2>"),
    ([800], 24, 16256, "grouped_pipe_kernel<{},4,2,2>"),
]


def kernel_of(sizes, N, K, bits, extra=0):
    return awq.awq_gemm_grouped_kernel(sum(sizes) + extra, len(sizes), N, K, bits).split(" ")[0]


def test_every_kernel_of_the_dispatch_is_among_the_tiles():
    for bits in (4, 3):
        seen = {awq.awq_gemm_grouped_kernel(R, E, N, K, bits).split(" ")[0]
                for E in (1, 5, 64) for N in (8, 1000, 30000) for K in (128, 4096, 8064, 8192, 16256, 16384, 24576, 65536, 131072)
                for R in (1, 4, 16, 100, 700, 5000, 40000)}
        assert seen == {k.format(bits) for *_, k in TILES}


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 3])
@pytest.mark.parametrize("case", range(len(TILES)))
def test_tiles(case, bits):
    sizes, N, K, kernel = TILES[case]
    note(f"tiles {kernel.format(bits)} sizes={sizes} N={N} K={K}")
    assert kernel_of(sizes, N, K, bits, 3) == kernel.format(bits)
    check_grouped(sizes, N, K, bits, seed=100 + case, extra=3)
    check_grouped(sizes, N, K, bits, seed=200 + case, gather=3, extra=3)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 3])
@pytest.mark.parametrize("gather", [None, 2])
def test_tiles_of_many_rows_with_input_scales(bits, gather):
    note(f"tiles scaled bits={bits} gather={gather}")
    check_grouped([900, 1, 300, 420], 136, 384, bits, seed=300, gather=gather, scaled=True, extra=3)
    check_grouped([900, 1, 1300, 420], 136, 384, bits, seed=301, gather=gather, scaled=True)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 3])
@pytest.mark.parametrize("K", [768, 8192, 11008])
def test_tiles_with_scales_of_zero_and_extremes(K, bits):
    """As for few rows: groups of scale 0 add nothing, scales of opposite extremes and signs follow one
    another, in two experts of 450 rows."""
    E, N, rows = 2, 70, 450
    assert kernel_of([rows] * E, N, K, bits).startswith(f"grouped_pipe_kernel<{bits},4,2,")
    g = np.random.default_rng(K + bits)
    _, p, sc, z = layer(E, N, K, bits, 9)
    s = host(sc).reshape(E * N, K // 128).copy()
    s[g.random(s.shape) < 0.3] = 0
    s[0], s[1, 0], s[2, -1] = 0, 0, 0
    s[3, ::2], s[3, 1::2] = 2.0 ** -14, 100.0
    s[4, ::2], s[4, 1::2] = -0.01, 0.02
    q = (decode_codes if bits == 4 else decode_codes3)(host(p).reshape(E * N, -1), K).astype(np.float64)
    zz = decode_zeros(host(z).reshape(E * N, -1), K // 128)
    w = ((q - np.repeat(zz, 128, 1)) * np.repeat(s.astype(np.float64), 128, 1)).reshape(E, N, K)
    x = inputs(E * rows, K, 10)
    y = host(awq.awq_gemm_grouped(dev(x), p, dev(s.reshape(E, N, -1)), z, dev(np.array([0, rows, 2 * rows], np.int32))))
    for e in range(E):
        assert_rows(y[e * rows:(e + 1) * rows], x[e * rows:(e + 1) * rows], w[e], f"expert {e}")
    assert np.all(y[:rows, 0] == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 3])
def test_tiles_with_an_infinite_input(bits):
    """An infinity stays in its own row, wherever the row stands in the tile."""
    N, K, at, rows = 50, 640, 600, 450
    w, p, sc, z = layer(2, N, K, bits, 31)
    x = inputs(2 * rows, K, 32)
    hit = [0, 40, 255, 256, rows - 1]
    x[hit, at] = np.inf
    y = host(awq.awq_gemm_grouped(dev(x), p, sc, z, dev(np.array([0, rows, 2 * rows], np.int32))))
    with np.errstate(invalid="ignore"):
        for i in hit:
            assert np.array_equal(y[i].astype(np.float64), np.inf * w[0, :, at], equal_nan=True)
    rest = np.setdiff1d(np.arange(rows), hit)
    assert_rows(y[rest], x[rest], w[0], "expert 0")
    assert_rows(y[rows:], x[rows:], w[1], "expert 1")


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(1, 1024, 1), (3, 1024, 64), (16, 1024, 64), (128, 1000, 8), (1024, 901, 1)])
def test_routes_and_plans_of_many_experts_in_one_launch(T, E, k):
    note(f"route T={T} E={E} k={k}")
    g = np.random.default_rng(T + E + k)
    x = g.standard_normal((T, E)).astype(np.float32)
    assert_route(awq.awq_moe_route(dev(x), k), x, k, True)
    experts = g.integers(-1, E + 1, size=(T, k)).astype(np.int32)
    experts[0, 0] = E - 1
    assert_plan(awq.awq_moe_plan(dev(experts), E), experts, E)
