"""Rows in 8 bits at the nearest quotients to a half that fp32 values can form.

For v = a 2^i and max|v| = b 2^(i+d), a and b whole and of 24 bits, 127 v / max|v| = 254 a / (2 b 2^d) differs from the half
h / 2 by (254 a - h 2^d b) / (2 b 2^d).  Pairs whose numerator is the smallest possible, +-2 (+-1 where d is 0), and 0 for a
half itself, are found here by whole-number arithmetic, so the wanted code is known without a rounding."""
import numpy as np
import pytest
import torch

import weight_only_quantization_gemm_amd as awq

DEV = "cuda:0"
STEP = 2.0 ** -10  # of the values: away from fp32's limits, also when they are squared


def pairs():
    """(v, max|v|, code) over every half h / 2 below 127, on both sides of it and on it."""
    found = [(8460799.0, 2149042944.0, 1)]  # 2^-31 above 1/2
    a = np.arange(1 << 23, (1 << 23) + (1 << 17), dtype=np.int64)  # the remainder takes every value among so many
    for h in range(1, 254, 2):
        d = int(np.floor(np.log2(254.0 / h)))
        step = h << d
        b = (254 * a + step // 2) // step
        left = 254 * a - step * b
        fits = (b >= 1 << 23) & (b < 1 << 24)
        for r in ((-2, 0, 2) if d > 0 else (-1, 0, 1)):
            at = np.flatnonzero(fits & (left == r))
            if at.size:
                i = at[at.size // 2]
                code = (h + 1) // 2 if r > 0 or (r == 0 and (h + 1) // 2 % 2 == 0) else (h - 1) // 2
                found.append((float(a[i]), float(b[i] << d), code))
    return found


PAIRS = pairs()


def test_pairs_are_the_nearest_there_are():
    """Every half has one on each side, their distance is from 2^-32 on (and 127 2^-53, the error of a quotient in
    64 bits, is far below it), and the values are fp32's."""
    assert len(PAIRS) >= 2 * 127
    least = min(abs(254 * int(v) - (2 * code - 1) * int(top)) / (2 * top) for v, top, code in PAIRS
                if 254 * int(v) != (2 * code - 1) * int(top))
    assert 2.0 ** -32 <= least <= 2.0 ** -31 * 1.001
    for v, top, code in PAIRS:
        assert np.float32(v) == v and np.float32(top) == top and v < top
        assert 2 * code * int(top) - int(top) <= 254 * int(v) <= 2 * code * int(top) + int(top)
        assert code == np.rint(127.0 * v / top)  # 64 bits decide them


def rows(n):
    """A row for each pair: its largest value, then v and -v, and smaller values."""
    x = np.zeros((len(PAIRS), n), np.float64)
    want = np.zeros((len(PAIRS), n), np.int64)
    for i, (v, top, code) in enumerate(PAIRS):
        x[i, :4] = v, -v, top, -v
        want[i, :4] = code, -code, 127, -code
    return (x * STEP).astype(np.float32), want


@pytest.mark.gpu
@pytest.mark.parametrize("n", [8, 1032])
def test_norm_of_an_fp32_stream(n):
    x, want = rows(n)
    one = torch.ones(n, dtype=torch.float16, device=DEV)
    r = awq.awq_norm(torch.from_numpy(x).to(DEV), one, quantize=True)
    assert np.array_equal(r["x"].cpu().numpy(), want)


@pytest.mark.gpu
def test_weights_times_s():
    x, want = rows(128)
    one = torch.ones(1, 128, dtype=torch.float16, device=DEV)
    for i in range(0, len(PAIRS), 7):
        codes, scales = awq.awq_pack_i8(one, torch.from_numpy(x[i]).to(DEV))
        assert np.array_equal(codes.cpu().numpy()[0], want[i])
        assert scales.item() == x[i].max() / np.float32(127)
