"""The grouped product with input scales: x / s enters with 22 bits up to five rows an expert (or 16
rows, and at most 2048), and rounded to fp16 as awq_scale_input rounds it beyond."""
import numpy as np
import pytest
import torch

import weight_only_quantization_gemm_amd as awq
from test_gpu_experts import DEV, dev, host, inputs, layer, note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gather", [0, 3])
@pytest.mark.parametrize("bits", [4, 3])
@pytest.mark.parametrize("sizes,K", [([1, 0, 2], 256), ([9, 7], 128), ([3, 9, 0, 8, 11, 1, 4, 4], 640),
                                     ([0, 0, 17, 1, 0, 2], 1408), ([2] * 1024, 128)])
def test_scaled_input_of_one_channel_keeps_22_bits(sizes, K, bits, gather):
    """Rows of one channel each: y is x / s times one weight, with no sum to blur it.  Off by the
    rounding of y (half a step: 2^-11 of it), by 2^-22 of x / s as two fp16 numbers (of 0.5 to 8
    here: the second is off by at most 2^-25 where it is no normal number), by the fp32 division,
    the group scale's product and the addition of the two (2^-24 each).  x / s rounded to fp16
    would be off by up to 2^-11 more."""
    E, R, N = len(sizes), sum(sizes), 72
    note(f"scaled E={E} R={R} K={K} bits={bits} gather={gather}")
    w, p, sc, z = layer(E, N, K, bits, 60)
    g = np.random.default_rng(R + K + bits)
    M = -(-R // gather) if gather else R
    at = g.integers(0, K, size=M)
    x = np.zeros((M, K), np.float16)
    x[np.arange(M), at] = g.uniform(1, 4, M) * np.where(g.random(M) < 0.5, -1, 1)
    s = np.exp2(g.uniform(-1, 1, (E, K))).astype(np.float32)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    kw, row = dict(s=dev(s)), np.arange(R)
    if gather:
        rows = g.permutation(R).astype(np.int32)
        kw.update(rows=dev(rows), top_k=gather)
        row = rows // gather
    out = torch.full((R + 1, N), 7.0, dtype=torch.float16, device=DEV)
    y = host(awq.awq_gemm_grouped(dev(x), p, sc, z, dev(offsets), out=out[:R], **kw)).astype(np.float64)
    assert np.all(host(out)[R] == 7.0)
    e = np.repeat(np.arange(E), sizes)
    ref = (x[row, at[row]].astype(np.float64) / s[e, at[row]])[:, None] * w[e, :, at[row]]
    bad = np.abs(y - ref) > (2.0 ** -11 + 2.0 ** -22 + 4 * 2.0 ** -24) * np.abs(ref) + 2.0 ** -25
    assert not bad.any(), (int(bad.sum()), bad.size)


@pytest.mark.parametrize("E,R", [(1, 16), (4, 20), (60, 300), (1024, 2048)])
def test_scaled_input_of_more_rows_is_rounded_as_the_single_products_is(E, R):
    """With one row more the scaled product is the product of fp16(x / s), bit for bit."""
    N, K = 40, 256
    _, p, sc, z = layer(E, N, K, 4, 61)
    g = np.random.default_rng(E)
    s = np.exp(0.4 * g.standard_normal((E, K))).astype(np.float32)
    for n in (R, R + 1):
        x = inputs(n, K, 62)
        off = np.concatenate([[0], np.sort(g.integers(0, n + 1, size=E - 1)), [n]]).astype(np.int32)
        e = np.repeat(np.arange(E), np.diff(off))
        y = host(awq.awq_gemm_grouped(dev(x), p, sc, z, dev(off), s=dev(s)))
        rounded = (x.astype(np.float32) / s[e]).astype(np.float16)
        same = np.array_equal(y.view(np.uint16), host(awq.awq_gemm_grouped(dev(rounded), p, sc, z, dev(off))).view(np.uint16))
        assert same == (n > R)
