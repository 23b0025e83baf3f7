"""Rows in 8 bits and awq_gemm_i8 against whole-number products.

The codes are compared exactly (their definition has one value); the sums are exact in 32 bits, so a
result is off by its roundings alone: the sum to fp32, two scales, and fp16 where that is the type
(2^-24 each of the first three, 2^-11 the last, 2^-25 among fp16's subnormals)."""
import numpy as np
import pytest
import torch

import weight_only_quantization_gemm_amd as awq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def codes_of(v):
    """Codes and scales of rows v (float32), exactly: 53 bits hold 127 v / max|v| well enough that
    no half is missed or made."""
    v = v.astype(np.float64)
    top = np.abs(v).max(1)
    return (np.rint(127 * v / np.where(top > 0, top, 1)[:, None]).astype(np.int8),
            (top.astype(np.float32) / np.float32(127)))


def rows(M, K, seed):
    g = np.random.default_rng(seed)
    x = g.standard_normal((M, K)) * np.exp(g.standard_normal((M, 1))) * np.where(g.random(K) < 0.02, 10, 1)
    return x.astype(np.float16)


def weights(N, K, seed):
    g = np.random.default_rng(seed)
    return g.integers(-127, 128, (N, K)).astype(np.int8), np.exp(g.standard_normal(N)).astype(np.float32) * 1e-4


def product(xc, xs, wc, ws):
    whole = xc.astype(np.float64) @ wc.astype(np.float64).T  # below 2^31: exact
    return whole * xs.astype(np.float64)[:, None] * ws.astype(np.float64)


def close(got, want):
    tol = 3.1 * 2.0 ** -24 * np.abs(want)
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -11 * np.abs(want) * (1 + 2.0 ** -20) + 2.0 ** -25
    bad = ~(np.abs(got.double().cpu().numpy() - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])


def dev(*arrays):
    return [torch.from_numpy(a).to(DEV) for a in arrays]


@pytest.mark.parametrize("M,K", [(1, 128), (3, 256), (2, 1408), (5, 4096), (2, 11008), (3, 32768), (1, 131072), (400, 384)])
@pytest.mark.parametrize("scaled", [False, True])
def test_quantize_rows(M, K, scaled):
    x = rows(M, K, seed=K)
    x[M // 2] = 0 if M > 1 else x[0]
    s = np.exp(0.5 * np.random.default_rng(1).standard_normal(K)).astype(np.float32) if scaled else None
    v = x.astype(np.float32) / s if scaled else x.astype(np.float32)
    want, scales = codes_of(v)
    codes, got = awq.awq_quantize_rows(*dev(x), *(dev(s) if scaled else ()))
    assert np.array_equal(codes.cpu().numpy(), want) and np.array_equal(got.cpu().numpy(), scales)
    # rows of a wider matrix
    wide = torch.zeros(M, K + 40, dtype=torch.float16, device=DEV)
    wide[:, 8:8 + K] = torch.from_numpy(x).to(DEV)
    codes2, got2 = awq.awq_quantize_rows(wide[:, 8:8 + K], *(dev(s) if scaled else ()))
    assert torch.equal(codes, codes2) and torch.equal(got, got2)
    # weights are multiplied
    v = x.astype(np.float32) * s if scaled else v
    want, scales = codes_of(v)
    codes, got = awq.awq_pack_i8(*dev(x), *(dev(s) if scaled else ()))
    assert np.array_equal(codes.cpu().numpy(), want) and np.array_equal(got.cpu().numpy(), scales)


def test_codes_of_every_ratio_of_small_numbers():
    """v / max|v| over all pairs of whole numbers up to 1024: every half that can occur among them."""
    K = 1024
    x = np.tile(np.arange(K, dtype=np.float16), (K, 1))
    x = np.where(np.arange(K)[None, :] <= np.arange(K)[:, None], x, np.float16(0)) * np.where(np.arange(K) % 3, 1, -1).astype(np.float16)
    want, scales = codes_of(x.astype(np.float32))
    codes, got = awq.awq_quantize_rows(*dev(x))
    assert np.array_equal(codes.cpu().numpy(), want) and np.array_equal(got.cpu().numpy(), scales)


SHAPES = [(M, N, K) for M in (1, 2, 5, 8, 16, 17, 31, 32, 33, 64, 65, 96, 128, 130, 255, 257, 300)
          for N, K in ((1, 128), (33, 384), (130, 1024), (1000, 256))]
SHAPES += [(M, N, K) for M in (1, 3, 16, 48, 64, 200) for N, K in ((257, 4096), (96, 11008), (4097, 512), (16, 32768))]
SHAPES += [(513, 515, 640), (700, 300, 128), (1025, 768, 1408), (2048, 100, 256), (40, 20000, 256), (600, 6000, 256)]
SHAPES += [(77, 1001, 4096), (33, 515, 11008), (100, 259, 8192), (256, 1030, 4096), (8, 26001, 512), (50, 30000, 256),
           (300, 2050, 11008), (497, 4090, 1024), (3999, 4093, 512)]  # shares of K with odd channels, and wide layers of few tokens


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    x = rows(M, K, seed=M)
    wc, ws = weights(N, K, seed=N)
    xc, xs = codes_of(x.astype(np.float32))
    want = product(xc, xs, wc, ws)
    dx, dxc, dxs, dwc, dws = dev(x, xc, xs, wc, ws)
    print(awq.awq_gemm_i8_kernel(M, N, K), flush=True)
    for dtype in (torch.float16, torch.float32):
        given = awq.awq_gemm_i8(dxc, dwc, dws, x_scales=dxs, dtype=dtype)
        close(given, want)
        assert torch.equal(awq.awq_gemm_i8(dx, dwc, dws, dtype=dtype), given)  # quantised on the way


@pytest.mark.parametrize("M", [1, 7, 16, 50, 300])
def test_scaled_input(M):
    N, K = 200, 1408
    x = rows(M, K, seed=M)
    s = np.exp(np.random.default_rng(3).standard_normal(K)).astype(np.float32)
    wc, ws = weights(N, K, seed=N)
    xc, xs = codes_of(x.astype(np.float32) / s)
    dx, dwc, dws, dsv = dev(x, wc, ws, s)
    close(awq.awq_gemm_i8(dx, dwc, dws, s=dsv), product(xc, xs, wc, ws))


@pytest.mark.parametrize("M", [1, 16, 64, 257])
def test_largest_sum(M):
    """Every code +-127 at K = 2^17: sums of 127^2 2^17 = 2114060288, next to 2^31."""
    K, N = 1 << 17, 20
    sign = np.where(np.arange(N) % 2, 1, -1).astype(np.int8)
    xc, wc = np.full((M, K), 127, np.int8), np.repeat(127 * sign[:, None], K, 1)
    ones_m, ones_n = np.ones(M, np.float32), np.ones(N, np.float32)
    y = awq.awq_gemm_i8(*dev(xc, wc, ones_n), x_scales=dev(ones_m)[0], dtype=torch.float32)
    assert np.array_equal(y.cpu().numpy(), np.repeat((np.float32(2114060288) * sign.astype(np.float32))[None], M, 0))


@pytest.mark.parametrize("M,N,K", [(1, 300, 512), (9, 300, 512), (33, 300, 1024), (70, 300, 512), (300, 520, 512)])
def test_one_row_and_one_channel_at_a_time(M, N, K):
    """Unit rows: y is the weights' codes themselves, so a misplaced row, channel or k shows."""
    g = np.random.default_rng(M)
    at = g.integers(0, K, M)
    xc = np.zeros((M, K), np.int8)
    xc[np.arange(M), at] = 1
    wc, _ = weights(N, K, seed=K)
    y = awq.awq_gemm_i8(*dev(xc, wc, np.ones(N, np.float32)), x_scales=dev(np.ones(M, np.float32))[0])
    assert np.array_equal(y.cpu().numpy(), wc[:, at].T.astype(np.float16))


def test_outputs_and_workspaces_given():
    M, N, K = 40, 130, 512
    x = rows(M, K, seed=1)
    wc, ws = weights(N, K, seed=2)
    dx, dwc, dws = dev(x, wc, ws)
    want = awq.awq_gemm_i8(dx, dwc, dws, dtype=torch.float32)
    need = awq.awq_gemm_i8_workspace_bytes(M, N, K, False)
    out = torch.full((M, N), 7.0, device=DEV)
    ws_t = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # needs no clearing
    for _ in range(2):
        assert awq.awq_gemm_i8(dx, dwc, dws, out=out, workspace=ws_t) is out
        assert torch.equal(out, want)


@pytest.mark.parametrize("M", [1, 24, 80, 520])
def test_nothing_is_written_past_the_output(M):
    N, K = 201, 256
    x = rows(M, K, seed=1)
    wc, ws = weights(N, K, seed=2)
    dx, dwc, dws = dev(x, wc, ws)
    buf = torch.full((M * N + 4096,), 7.0, dtype=torch.float16, device=DEV)
    out = buf[:M * N].view(M, N)
    awq.awq_gemm_i8(dx, dwc, dws, out=out)
    assert torch.equal(buf[M * N:], torch.full((4096,), 7.0, dtype=torch.float16, device=DEV))
    assert torch.equal(out, awq.awq_gemm_i8(dx, dwc, dws))


@pytest.mark.parametrize("M,N,K", [(1, 1000, 1024), (24, 1000, 4096), (100, 500, 4096), (600, 512, 512)])
def test_other_stream_and_graph(M, N, K):
    x = rows(M, K, seed=1)
    wc, ws = weights(N, K, seed=2)
    dx, dwc, dws = dev(x, wc, ws)
    want = awq.awq_gemm_i8(dx, dwc, dws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = awq.awq_gemm_i8(dx, dwc, dws)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = awq.awq_gemm_i8(dx, dwc, dws)
    for _ in range(3):
        dx.mul_(-0.5)
        want = awq.awq_gemm_i8(dx, dwc, dws)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_refusals():
    x, (wc, ws) = rows(4, 256, seed=1), weights(8, 256, seed=2)
    dx, dwc, dws = dev(x, wc, ws)
    xc, xs = awq.awq_quantize_rows(dx)
    for bad in (lambda: awq.awq_gemm_i8(dx, dwc[:, :128].contiguous(), dws), lambda: awq.awq_gemm_i8(dx, dwc, dws[:4]),
                lambda: awq.awq_gemm_i8(xc, dwc, dws, x_scales=xs, s=torch.ones(256, device=DEV)),
                lambda: awq.awq_gemm_i8(xc, dwc, dws, x_scales=xs[:3]), lambda: awq.awq_gemm_i8(dx, dwc, dws.cpu()),
                lambda: awq.awq_gemm_i8(dx, dwc, dws, out=torch.empty(4, 7, device=DEV)),
                lambda: awq.awq_gemm_i8(dx[:, :200].contiguous(), dwc[:, :200].contiguous(), dws),
                lambda: awq.awq_quantize_rows(dx[:, :200]), lambda: awq.awq_pack_i8(dx[:, :128])):
        with pytest.raises((ValueError, awq.AwqError)):
            bad()
    for bad in (lambda: awq.awq_gemm_i8(xc, dwc, dws), lambda: awq.awq_gemm_i8(dx, dwc, dws, x_scales=xs),
                lambda: awq.awq_gemm_i8(dx, dwc, dws, dtype=torch.bfloat16),
                lambda: awq.awq_gemm_i8(dx, dwc, dws.half())):
        with pytest.raises(TypeError):
            bad()


@pytest.mark.parametrize("M,K", [(1, 256), (3, 4096), (1500, 4096), (5, 11008), (2, 20480)])
def test_rows_with_infinities_and_nan(M, K):
    """Such a row's codes are 0 and its scale is infinite or NaN, so its products are NaN; the other
    rows are as without it."""
    x = rows(M, K, seed=K)
    for value in (np.inf, -np.inf, np.nan):
        for at in (0, K // 2 + 5, K - 1):
            bad = x.copy()
            bad[M // 2, at] = value
            codes, scales = awq.awq_quantize_rows(*dev(bad))
            scales = scales.cpu().numpy()
            assert not codes[M // 2].any()
            assert np.isnan(scales[M // 2]) if np.isnan(value) else np.isposinf(scales[M // 2])
            want, want_scales = codes_of(np.delete(x, M // 2, 0).astype(np.float32)) if M > 1 else (x[:0], x[:0, 0])
            assert np.array_equal(np.delete(codes.cpu().numpy(), M // 2, 0), want)
            assert np.array_equal(np.delete(scales, M // 2), want_scales)
            wc, ws = weights(40, K, seed=1)
            y = awq.awq_gemm_i8(*dev(bad, wc, ws))
            assert y[M // 2].isnan().all() and not np.isnan(np.delete(y.cpu().numpy(), M // 2, 0)).any()
