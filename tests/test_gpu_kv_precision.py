"""The precision that attention over the low-bit cache states, where the other tests' tolerances
(worst cases of sums) leave room: against definitions in 64 bits (numpy)."""
import numpy as np
import pytest
import torch

import weight_only_quantization_gemm_amd as awq
from test_gpu_kv_cache import ORDER, attend_ref, host_cache, random_cache, unpack
from test_gpu_experts import DEV, dev, host, note

pytestmark = pytest.mark.gpu


def pack(codes, bits):
    """uint32 words (as int32) of codes [..., D]."""
    sh = [4 * o for o in ORDER] if bits == 4 else [0, 8, 16, 24]
    c = codes.astype(np.uint32).reshape(*codes.shape[:-1], -1, len(sh))
    return np.bitwise_or.reduce(c << np.array(sh, np.uint32), -1).astype(np.uint32).view(np.int32)


def bell_cache(n, D, bits, seed, page=16):
    """One head's cache of n tokens of bell-shaped keys and values of about unit size."""
    g = np.random.default_rng(seed)
    c = awq.empty_kv_cache(n // page, 1, D, page=page, bits=bits, device=DEV)
    zero, step = 2 ** (bits - 1), 6.0 / 2 ** bits
    for x in "kv":
        codes = np.clip(np.rint(g.standard_normal((n, D)) / step) + zero, 0, 2 ** bits - 1)
        c[x + "_codes"].copy_(dev(pack(codes, bits).reshape(c[x + "_codes"].shape)))
        scale = step * np.exp(0.1 * g.standard_normal(n))
        c[x + "_params"].copy_(dev(np.stack([scale, np.full(n, zero)], -1).astype(np.float16).reshape(-1, 1, page, 2)))
    return c


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_error_over_long_sequences_is_that_of_rounding_the_output(D, bits):
    """400000 tokens of no common direction: the output is some 500 times smaller than the values.
    Its rounding to fp16 is still the whole error: all that stands before it adds less than 1 %
    to the error's root mean square (so is below 14 % of it), and leaves no mean (5 standard
    deviations of that of the roundings).  By the statement: weights are off by 2^-22 each and
    independently, sums of a piece (up to 128 of a wave) by 2^-24 of about 128 steps of a value,
    over 400 pieces and waves: some 2 % of the rounding in all."""
    n, r = 400000, 16
    note(f"long D={D} bits={bits}")
    c = bell_cache(n, D, bits, 51)
    q = np.random.default_rng(52).standard_normal((1, r, D)).astype(np.float16)
    table = np.random.default_rng(53).permutation(n // 16)[None].astype(np.int32)
    y = host(awq.awq_kv_attention(dev(q), c, dev(table), dev(np.array([n], np.int32)))).astype(np.float64)[0]
    h = host_cache(c)
    kc, vc = (unpack(h[x + "_codes"][:, 0], bits).reshape(n, D).astype(np.float64) for x in "kv")
    kp, vp = (h[x + "_params"][:, 0].reshape(n, 2).astype(np.float64) for x in "kv")
    s = D ** -0.5 * (q[0].astype(np.float64) @ ((kc - kp[:, 1:]) * kp[:, :1]).T)
    p = np.exp(s - s.max(1, keepdims=True))
    out = (p / p.sum(1, keepdims=True)) @ ((vc - vp[:, 1:]) * vp[:, :1])
    rounding = np.sqrt(((out.astype(np.float16).astype(np.float64) - out) ** 2).mean())
    err = y - out
    note(f"rms error / rounding {np.sqrt((err ** 2).mean()) / rounding:.4f}, mean {err.mean() / rounding * np.sqrt(err.size):.2f} deviations")
    assert np.sqrt((err ** 2).mean()) <= 1.01 * rounding
    assert abs(err.mean()) <= 5 * rounding / np.sqrt(err.size)


def large_scores(n, D, bits, r, q_size, key_scale, scale, seed, winner=None):
    """One sequence of n tokens of equal keys (token `winner`'s scale twice theirs): output, and the
    definition's with the tolerance of its weights, which are equal or 0 and 1."""
    g = np.random.default_rng(seed)
    c = random_cache(n // 16 + 1, 1, D, 16, bits, seed)
    c["k_codes"].copy_(c["k_codes"][:1, :, :1].clone().expand_as(c["k_codes"]))
    c["k_params"][..., 0] = key_scale
    c["k_params"][..., 1] = 2 ** (bits - 1)
    kc = unpack(host(c["k_codes"])[0, 0, 0], bits) - 2.0 ** (bits - 1)
    q = np.minimum(np.abs(g.standard_normal((1, r, D))) * q_size + q_size / 4, 60000)
    q = (q * np.where(kc > 0, 1, -1) * np.sign(scale)).astype(np.float16)  # scores above 0
    if winner is not None:
        c["k_params"][winner // 16, 0, winner % 16, 0] = 2 * key_scale
    table = np.arange(n // 16 + 1, dtype=np.int32)[None]
    h = host_cache(c)
    s = scale * (q[0].astype(np.float64) @ kc) * key_scale
    assert np.all(np.isfinite(s)) and s.min() > 100  # twice the score: e^100 times the weight
    y = host(awq.awq_kv_attention(dev(q), c, dev(table), dev(np.array([n], np.int32)), scale=scale)).astype(np.float64)[0]
    at = np.arange(n) if winner is None else np.array([winner])
    vc = unpack(h["v_codes"][at // 16, 0, at % 16], bits).astype(np.float64)
    vp = h["v_params"][at // 16, 0, at % 16].astype(np.float64)
    ref, mag = ((vc - vp[:, 1:]) * vp[:, :1]).mean(0), ((vc + vp[:, 1:]) * vp[:, :1]).mean(0)
    return y, ref, 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (64 + n // 128) * 2.0 ** -22 * mag, s


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n,winner", [(1, None), (40, None), (40, 17), (700, None), (700, 699), (6000, None), (6000, 3001)])
def test_large_scores_weigh_tokens_as_small_ones_do(n, winner, bits):
    """Scores of 2^12 to 2^90: equal ones share the output, the largest one takes it, in one piece and
    in several.  Large queries and keys at the default scale, and ordinary ones at large scales."""
    D, r = 128, 3
    for size, key, scale in ((4.0, 2.0, D ** -0.5), (300.0, 20.0, D ** -0.5), (20000.0, 3000.0, D ** -0.5),
                             (20000.0, 8000.0, -1.0), (1.0, 0.1, 1e12), (1.0, 0.1, -2.0 ** 64), (20000.0, 8000.0, 2.0 ** 64),
                             (0.01, 0.001, 2.0 ** 40)):
        y, ref, tol, s = large_scores(n, D, bits, r, size, key, scale, 71, winner)
        note(f"scores of 2^{np.log2(s.max()):.1f}")
        assert np.all(np.abs(y - ref) <= tol), (size, key, scale, y[0, :4], ref[:4])


def test_large_scores_in_pieces_of_ragged_sequences():
    """A batch split by the lengths, scores of 2^40 and more: each sequence of equal keys gives its mean."""
    g = np.random.default_rng(72)
    lengths = np.array([5000, 0, 1, 129, 2600, 17], np.int32)
    D, page = 64, 16
    c = random_cache(700, 2, D, page, 4, 73)
    c["k_codes"].copy_(c["k_codes"][:1, :, :1].clone().expand_as(c["k_codes"]))
    c["k_params"][..., 0] = 4000.0
    c["k_params"][..., 1] = 7
    table = g.permutation(700)[:600].reshape(6, 100)
    table = np.concatenate([table, g.integers(0, 700, size=(6, 400))], 1).astype(np.int32)
    q = (g.standard_normal((6, 8, D)) * 8000).astype(np.float16)
    y = host(awq.awq_kv_attention(dev(q), c, dev(table), dev(lengths), scale=2.0 ** 10)).astype(np.float64)
    h = host_cache(c)
    for b, n in enumerate(lengths):
        t = np.arange(n)
        for k in range(2):
            if n == 0:
                assert np.all(y[b] == 0)
                continue
            vc = unpack(h["v_codes"][table[b, t // page], k, t % page], 4).astype(np.float64)
            vp = h["v_params"][table[b, t // page], k, t % page].astype(np.float64)
            ref, mag = ((vc - vp[:, 1:]) * vp[:, :1]).mean(0), ((vc + vp[:, 1:]) * vp[:, :1]).mean(0)
            tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (64 + n // 128) * 2.0 ** -22 * mag
            assert np.all(np.abs(y[b, 4 * k:4 * k + 4] - ref) <= tol)


def one_channel_scores(steps, scale_of_values, D, bits, seed):
    """One sequence whose scores are known: q is 1 in channel 0, a key's code there `steps` (a token's,
    whole) from its zero point, its scale 2^-4, the attention's scale 1: score steps / 16, exactly.
    Values: random codes, the given scales.  Returns the output, the definition's weights, values and
    the values' magnitudes (code + zero) scale."""
    n = len(steps)
    c = random_cache(-(-n // 16), 1, D, 16, bits, seed)
    kw = np.full((c["k_codes"].shape[0] * 16, D), 2 ** (bits - 1))
    kw[:n, 0] += steps
    assert kw.min() >= 0 and kw.max() < 2 ** bits
    c["k_codes"].copy_(dev(pack(kw, bits).reshape(c["k_codes"].shape)))
    c["k_params"][..., 0] = 2.0 ** -4
    c["k_params"][..., 1] = 2 ** (bits - 1)
    vs = np.ones(kw.shape[0])
    vs[:n] = scale_of_values
    c["v_params"][..., 0] = dev(vs.reshape(-1, 1, 16).astype(np.float16))
    q = np.zeros((1, 1, D), np.float16)
    q[0, 0, 0] = 1
    table = np.arange(kw.shape[0] // 16, dtype=np.int32)[None]
    y = host(awq.awq_kv_attention(dev(q), c, dev(table), dev(np.array([n], np.int32)), scale=1.0)).astype(np.float64)[0, 0]
    h, t = host_cache(c), np.arange(n)
    vc = unpack(h["v_codes"][t // 16, 0, t % 16], bits).astype(np.float64)
    vp = h["v_params"][t // 16, 0, t % 16].astype(np.float64)
    p = np.exp(np.asarray(steps) / 16.0)
    return y, p / p.sum(), (vc - vp[:, 1:]) * vp[:, :1], (vc + vp[:, 1:]) * vp[:, :1]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [2, 3, 17, 300])
def test_weights_enter_with_22_bits(n, D, bits):
    """Scores are exact here, so that the weights show: exp2's argument rounds twice (2^-23 of at most
    0.7: 2^-23 of the weight), exp2 and the value scale's product once each, two fp16 numbers leave
    2^-22: 2^-20.9 in all; sums of at most 10 steps, waves and products in fp32, 2^-19.5 of the
    magnitudes.  Weights of one fp16 number (2^-12) are seen, where there are enough for their
    roundings not to be small by chance: the bound refuses them."""
    g = np.random.default_rng(n + D + bits)
    steps = g.integers(-8, 8, size=n) if bits == 4 else g.integers(-11, 12, size=n)
    vs = np.exp(0.5 * g.standard_normal(n)).astype(np.float16)
    y, p, v, mag = one_channel_scores(steps, vs, D, bits, 81 + n)
    ref = p @ v
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2.0 ** -19 * (p @ mag)
    assert bool(np.all(np.abs(y - ref) <= tol))
    w = p * vs.astype(np.float64)
    once = (w / w.max() * 100).astype(np.float16).astype(np.float64) * w.max() / 100 / vs.astype(np.float64)
    assert n < 17 or bool(np.any(np.abs(once @ v - ref) > tol))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n,wide", [(40, 0), (40, 39), (300, 150), (700, 3), (4000, 0), (4000, 3999)])
def test_a_large_value_of_no_weight_leaves_the_others_their_bits(n, wide, bits):
    """One token's value scale is the largest that is written (of a row from -65504 to 65504), all
    others' the smallest, and its weight e^-60: the others' weights keep their 22 bits."""
    D = 64
    g = np.random.default_rng(n + wide + bits)
    steps = g.integers(-8, 8, size=n) if bits == 4 else g.integers(-64, 0, size=n)
    vs = np.full(n, 2.0 ** -14, np.float16)
    vs[wide] = np.float16(131008 / (2 ** bits - 1))
    # the scores' range is 0.5 .. 4 here; the wide token's is pushed down by its key's own scale
    c = random_cache(-(-n // 16), 1, D, 16, bits, 91)
    kw = np.full((c["k_codes"].shape[0] * 16, D), 2 ** (bits - 1))
    kw[:n, 0] += steps
    kw[wide, 0] = 0
    c["k_codes"].copy_(dev(pack(kw, bits).reshape(c["k_codes"].shape)))
    ks = np.full(kw.shape[0], 2.0 ** -4)
    ks[wide] = 64 / 2.0 ** (bits - 1)
    c["k_params"][..., 0] = dev(ks.reshape(-1, 1, 16).astype(np.float16))
    c["k_params"][..., 1] = 2 ** (bits - 1)
    full = np.ones(kw.shape[0])
    full[:n] = vs
    c["v_params"][..., 0] = dev(full.reshape(-1, 1, 16).astype(np.float16))
    q = np.zeros((1, 1, D), np.float16)
    q[0, 0, 0] = 1
    table = np.arange(kw.shape[0] // 16, dtype=np.int32)[None]
    y = host(awq.awq_kv_attention(dev(q), c, dev(table), dev(np.array([n], np.int32)), scale=1.0)).astype(np.float64)[0, 0]
    h, t = host_cache(c), np.arange(n)
    vc = unpack(h["v_codes"][t // 16, 0, t % 16], bits).astype(np.float64)
    vp = h["v_params"][t // 16, 0, t % 16].astype(np.float64)
    s = np.where(t == wide, -64.0, steps / 16.0)
    p = np.exp(s - s.max())
    p /= p.sum()
    ref, mag = p @ ((vc - vp[:, 1:]) * vp[:, :1]), p @ ((vc + vp[:, 1:]) * vp[:, :1])
    assert p[wide] * 131008 < 1e-4 * mag.min()
    # exp2's argument of up to 2^2.6 rounds by 2^-21; sums of up to 64 steps, waves and pieces
    assert bool(np.all(np.abs(y - ref) <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2.0 ** -18 * mag))


@pytest.mark.parametrize("bits", [4, 8])
def test_value_scales_that_grow_and_fall_along_a_sequence(bits):
    """Value scales over the whole range that is written, in random order and in runs, with weights
    that rise and fall: the exponent that the weights share moves up and down."""
    D, n = 64, 3000
    g = np.random.default_rng(95)
    top = np.log2(131008 / (2 ** bits - 1))
    for vs in (np.exp2(g.uniform(-14, top, n)), np.exp2(-14 + (top + 14) * np.abs(np.sin(np.arange(n) / 200.0))),
               np.exp2(np.where(np.arange(n) % 64 < 32, -14, top)), np.exp2(np.linspace(top, -14, n))):
        steps = g.integers(-8, 8, size=n) if bits == 4 else (110 * np.sin(np.arange(n) / 317.0)).astype(int)
        y, p, v, mag = one_channel_scores(steps, vs.astype(np.float16), D, bits, 96)
        ref = p @ v
        # exp2's argument of up to 2^4.4 rounds by 2^-19.6
        tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2.0 ** -17.5 * (p @ mag)
        near = (np.abs(y - ref) <= tol) | ((y == np.copysign(np.inf, ref)) & (np.abs(ref) + tol >= 65520))
        assert near.all()


def test_many_heads_of_sequences_of_several_pieces():
    """64 heads, a few sequences of 20000 tokens among short and empty ones: pieces of more than one
    window of pages, joined for every head (three heads are checked)."""
    H, D, page, heads = 64, 64, 16, [0, 31, 63]
    g = np.random.default_rng(97)
    lengths = g.integers(0, 300, size=12).astype(np.int32)
    lengths[[0, 5, 11]] = [20000, 19999, 18433]
    lengths[3] = 0
    table = g.integers(0, 1500, size=(12, 1250)).astype(np.int32)  # pages shared between sequences
    c = random_cache(1500, H, D, page, 4, 98)
    q = g.standard_normal((12, H, D)).astype(np.float16)
    y = host(awq.awq_kv_attention(dev(q), c, dev(table), dev(lengths)))
    # units of 128 tokens of 64 heads, 1536 pieces of which fill the chip: pieces of 32 units, four windows
    units = int(np.maximum(1, -(-lengths // 128)).sum())
    assert 16 * 1536 < units * H <= 32 * 1536 and lengths[0] > 4 * 32 * 128
    sub = {k: v[:, heads] for k, v in host_cache(c).items()}
    ref, tol = attend_ref(q[:, heads], sub, table, lengths, D ** -0.5, 4, 160)
    assert bool(np.all(np.abs(y[:, heads] - ref) <= tol))
    assert np.all(y[3] == 0)


def test_a_cache_without_heads_is_refused():
    c = awq.empty_kv_cache(2, 0, 64, device=DEV)
    i = torch.zeros(1, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="heads"):
        awq.awq_kv_attention(torch.zeros(1, 2, 64, dtype=torch.float16, device=DEV), c, i[:, None].contiguous(), i)
