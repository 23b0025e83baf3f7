"""The low-bit key-value cache and attention over it, against plain implementations (numpy):
codes, scales and zero points bit for bit, attention in 64 bits.

Attention's tolerance (per query head, from the statement of its arithmetic): a score is a sum
of D products in fp32 on codes and zero points, off by at most D 2^-23 of the sum of their
magnitudes; that difference d moves every weight by a factor within e^(2 d); weights enter with
2^-22, exp2 with 2 ulp; sums over the tokens are at most 64 + chunks additions deep; the output
is rounded to fp16 once (2^-11)."""
import numpy as np
import pytest
import torch

import weight_only_quantization_gemm_amd as awq
from test_gpu_experts import DEV, dev, host, note

pytestmark = pytest.mark.gpu

ORDER = [0, 4, 1, 5, 2, 6, 3, 7]  # nibble of channel i of a word


def unpack(words, bits):
    w = np.ascontiguousarray(words).view(np.uint32)
    sh = [4 * o for o in ORDER] if bits == 4 else [0, 8, 16, 24]
    c = np.stack([(w >> np.uint32(s)) & np.uint32(2 ** bits - 1) for s in sh], -1)
    return c.reshape(*w.shape[:-1], -1).astype(np.int64)


def quantise(v, bits):
    """codes, scale (fp16), zero of rows [..., D], in the float32 arithmetic of the statement."""
    v = v.astype(np.float32)
    top = np.float32(2 ** bits - 1)
    lo, hi = np.minimum(v.min(-1), np.float32(0)), np.maximum(v.max(-1), np.float32(0))
    scale = np.maximum((hi - lo) / top, np.float32(2.0 ** -14)).astype(np.float16)
    s = scale.astype(np.float32)
    zero = np.clip(np.rint(-lo / s), 0, top)
    return np.clip(np.rint(v / s[..., None]) + zero[..., None], 0, top).astype(np.int64), scale, zero


def host_cache(c):
    return {k: host(v) for k, v in c.items() if k != "bits"}


def random_cache(pages, H, D, page, bits, seed, magnitude=0.3):
    g = np.random.default_rng(seed)
    c = awq.empty_kv_cache(pages, H, D, page=page, bits=bits, device=DEV)
    for x in "kv":
        shape = tuple(c[x + "_codes"].shape)
        c[x + "_codes"].copy_(dev(g.integers(0, 2 ** 32, size=shape, dtype=np.uint64).astype(np.uint32).view(np.int32)))
        zero = g.integers(2 ** (bits - 1) - 2, 2 ** (bits - 1) + 3, size=shape[:3])
        scale = magnitude / 2 ** (bits - 4) * np.exp(0.4 * g.standard_normal(shape[:3]))
        c[x + "_params"].copy_(dev(np.stack([scale, zero], -1).astype(np.float16)))
    return c


# ------------------------------------------------------------------ write, read
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,H,page", [(1, 1, 16), (5, 3, 16), (70, 2, 64), (33, 8, 1024)])
def test_write_and_read(T, H, page, D, bits):
    note(f"kv write T={T} H={H} page={page} D={D} bits={bits}")
    g = np.random.default_rng(T + H + D + bits)
    pages = -(-T // page) + 2
    c = random_cache(pages, H, D, page, bits, 1)
    before = host_cache(c)
    qkv = (g.standard_normal((T, 2 + 2 * H, D)) * np.exp(g.standard_normal((T, 2 + 2 * H, 1)))).astype(np.float16)
    qkv[0, 2] = 0                                        # a row of zeros
    qkv[T // 2, 2, :] = np.abs(qkv[T // 2, 2, :])        # of one sign
    qkv[-1, -1, :] = -np.abs(qkv[-1, -1, :]) * np.float16(1e-4)  # negative, tiny: the smallest scale
    qkv[-1, 2, 3], qkv[-1, 2, 5] = 65504, -65504         # the whole range of fp16
    slots = g.permutation(pages * page)[:T].astype(np.int32)
    if T > 4:
        slots[[1, 3]] = [-1, pages * page]               # padding: not written
    t = dev(qkv)
    awq.awq_kv_write(t[:, 2:2 + H], t[:, 2 + H:], dev(slots), c)
    after = host_cache(c)
    kr, vr = awq.awq_kv_read(c, dev(slots), D)
    written = (slots >= 0) & (slots < pages * page)
    for x, rows, back in (("k", qkv[:, 2:2 + H], kr), ("v", qkv[:, 2 + H:], vr)):
        codes, scale, zero = quantise(rows, bits)
        pg, at = slots // page, slots % page
        for i in np.flatnonzero(written):
            assert np.array_equal(unpack(after[x + "_codes"][pg[i], :, at[i]], bits), codes[i])
            assert np.array_equal(after[x + "_params"][pg[i], :, at[i], 0].view(np.uint16), scale[i].view(np.uint16))
            assert np.array_equal(after[x + "_params"][pg[i], :, at[i], 1], zero[i].astype(np.float16))
        value = ((codes - zero[..., None]) * scale.astype(np.float64)[..., None]).astype(np.float16)
        value[~written] = 0
        assert np.array_equal(host(back), value)
        # every other slot as it was
        other = np.ones(pages * page, bool)
        other[slots[written]] = False
        for n in (x + "_codes", x + "_params"):
            a, b = (v[n].transpose(0, 2, 1, 3).reshape(pages * page, -1)[other] for v in (before, after))
            assert np.array_equal(a.view(np.uint8), b.view(np.uint8))


def test_write_error_is_within_half_a_step():
    g = np.random.default_rng(0)
    x = g.standard_normal((40, 2, 128)).astype(np.float16)
    for bits in (4, 8):
        c = awq.empty_kv_cache(3, 2, 128, bits=bits, device=DEV)
        slots = dev(np.arange(40, dtype=np.int32))
        awq.awq_kv_write(dev(x), dev(-x), slots, c)
        k, v = awq.awq_kv_read(c, slots, 128)
        p = host(c["k_params"]).transpose(0, 2, 1, 3).reshape(48, 2, 2)[:40, :, 0].astype(np.float64)
        # half a step, one more where the rounded range or zero point clips, and the fp16 rounding of the value
        err = np.abs(host(k).astype(np.float64) - x)
        assert np.all(err <= p[..., None] * 1.01 + 2.0 ** -11 * np.abs(x))
        assert np.mean(err <= p[..., None] * 0.5 + 2.0 ** -11 * np.abs(x)) > 0.98


def test_write_non_finite_rows_stay_in_the_format():
    """Outside the contract: such a row's own codes are unspecified, nothing else changes."""
    x = np.ones((3, 1, 64), np.float16)
    x[1, 0, 5], x[1, 0, 6], x[1, 0, 7] = np.nan, np.inf, -np.inf
    c = random_cache(1, 1, 64, 16, 4, 2)
    awq.awq_kv_write(dev(x), dev(x), dev(np.array([2, 5, 7], np.int32)), c)
    k, _ = awq.awq_kv_read(c, dev(np.array([2, 7], np.int32)), 64)
    codes, scale, zero = quantise(x[0, 0], 4)
    assert np.all(host(k) == ((codes - zero) * scale.astype(np.float64)).astype(np.float16))


# -------------------------------------------------------------------- attention
def attend_ref(q, c, table, lengths, scale, bits, chunks):
    """out (fp64) and its tolerance; a sequence's tokens of bad pages are left out."""
    B, Hq, D = q.shape
    pages, H, page = c["k_codes"].shape[:3]
    r = Hq // H
    out, tol = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    for b in range(B):
        n = min(int(lengths[b]), table.shape[1] * page)
        t = np.arange(max(n, 0))
        pg = table[b, t // page] if n > 0 else t
        t = t[(pg >= 0) & (pg < pages)]
        if t.size == 0:
            continue
        pg, at = table[b, t // page], t % page
        for h in range(H):
            kc, vc = (unpack(c[x + "_codes"][pg, h, at], bits).astype(np.float64) for x in "kv")
            kp, vp = (c[x + "_params"][pg, h, at].astype(np.float64) for x in "kv")
            qh = q[b, h * r:(h + 1) * r].astype(np.float64)
            s = scale * (qh @ kc.T - qh.sum(1, keepdims=True) * kp[:, 1]) * kp[:, 0]
            ds = abs(scale) * D * 2.0 ** -23 * (np.abs(qh) @ (kc + kp[:, 1:]).T * kp[:, 0]).max(1) + 2.0 ** -22 * np.abs(s).max(1)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            o = p @ ((vc - vp[:, 1:]) * vp[:, :1])
            mag = p @ ((vc + vp[:, 1:]) * vp[:, :1])
            out[b, h * r:(h + 1) * r] = o
            tol[b, h * r:(h + 1) * r] = 2.0 ** -11 * np.abs(o) + 2.0 ** -25 + \
                (2 * ds[:, None] + (64 + chunks) * 2.0 ** -22) * mag
    return out, tol


def check_attention(B, lengths, H, r, D, page, bits, seed, scale=None, table=None, width=None, magnitude=0.3, q_gain=1.0,
                    max_len=0):
    g = np.random.default_rng(seed)
    lengths = np.asarray(lengths, np.int32)
    width = width or max(1, -(-int(max(lengths.max(), 1)) // page))
    pages = B * width + 2
    c = random_cache(pages, H, D, page, bits, seed + 1, magnitude)
    if table is None:
        table = g.permutation(pages)[:B * width].reshape(B, width).astype(np.int32)
    # what lies behind a length is never used: not the entries, not the slots (those of no sequence are NaN)
    live = np.zeros((pages, page), bool)
    for b in range(B):
        used = max(0, -(-int(lengths[b]) // page))
        table[b, used:] = np.iinfo(np.int32).max
        for t in range(max(0, int(lengths[b]))):
            if 0 <= table[b, t // page] < pages:
                live[table[b, t // page], t % page] = True
    dead = dev(~live)[:, None, :, None]
    for x in "kv":
        c[x + "_params"].masked_fill_(dead, float("nan"))
    fused = (g.standard_normal((B, H * (r + 2), D)) * q_gain).astype(np.float16)
    q = dev(fused)[:, :H * r]
    out = torch.full((B, H * r, D), 7.0, dtype=torch.float16, device=DEV)
    y = host(awq.awq_kv_attention(q, c, dev(table), dev(lengths), scale=scale, out=out, max_len=max_len))
    chunks = -(-width * page // 128)
    bound = np.minimum(lengths, max_len) if max_len else lengths
    ref, tol = attend_ref(fused[:, :H * r], host_cache(c), table, bound, D ** -0.5 if scale is None else scale, bits, chunks)
    bad = ~(np.abs(y.astype(np.float64) - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.abs(y - ref).max()))
    again = host(awq.awq_kv_attention(q, c, dev(table), dev(lengths), scale=scale, max_len=max_len))
    assert np.array_equal(again.view(np.uint16), y.view(np.uint16))
    return y, ref


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,r", [(1, 1), (2, 4), (3, 8), (1, 16), (2, 5), (1, 23)])
def test_attention_heads(H, r, D, bits):
    note(f"attention H={H} r={r} D={D} bits={bits}")
    check_attention(3, [77, 1, 300], H, r, D, 16, bits, seed=H + r + D + bits)


@pytest.mark.parametrize("page", [16, 32, 128, 1024])
@pytest.mark.parametrize("lengths", [[0], [1], [15, 16, 17], [31, 32, 33, 0, 64], [127, 128, 129, 2], [0, 0],
                                     [1000, 3, 1025, 512], [-4, 5], [2049, 4100]])
def test_attention_lengths(lengths, page):
    """Lengths of 0 and 1, ends inside and at pages, steps and chunks; what lies behind a length
    is NaN and bad pages.  A sequence with no tokens gives 0."""
    note(f"attention lengths={lengths} page={page}")
    y, _ = check_attention(len(lengths), lengths, 2, 4, 128, page, 4, seed=sum(lengths) + page)
    for b, n in enumerate(lengths):
        if n <= 0:
            assert np.all(y[b] == 0)


def test_attention_many_sequences_take_larger_chunks():
    check_attention(150, np.random.default_rng(3).integers(0, 2100, size=150), 8, 1, 64, 16, 4, seed=8)


def test_attention_many_long_sequences_take_the_largest_chunks():
    """Pieces whose pages are read in several runs of 1024 tokens; for more than 1024
    sequences chunks of 4096 tokens and a second one behind them."""
    n = np.random.default_rng(16).integers(2500, 4400, size=120)
    n[:4] = [4096, 4097, 4111, 0]
    check_attention(120, n, 8, 1, 64, 16, 4, seed=17)
    n = np.random.default_rng(27).integers(0, 300, size=1030)
    n[[5, 100, 101, 1029]] = [4400, 4096, 4097, 1025]
    check_attention(1030, n, 1, 2, 64, 16, 4, seed=28)


@pytest.mark.parametrize("B", [1, 3, 64, 65, 255, 256, 257, 513, 1024, 1025])
def test_attention_bound_far_above_the_lengths(B):
    """A page table made for 70000 tokens and sequences of a few hundred, some empty: the tokens
    are shared out by the lengths, up to 1024 sequences."""
    n = np.random.default_rng(B).integers(-100, 700, size=B)
    n[0] = 900
    check_attention(B, n, 2, 4, 64, 16, 4, seed=20 + B, width=4400 if B < 10 else 60)


def test_attention_runs_past_the_blocks():
    """More tokens than the blocks of a head take in one run each: they go on to further runs of
    4096 tokens (three of the 64 heads are checked)."""
    H, B, D, page, heads = 64, 40, 64, 16, [0, 31, 63]
    g = np.random.default_rng(23)
    lengths = g.integers(2000, 3000, size=B).astype(np.int32)
    lengths[[3, 17]] = [0, 1]
    table = g.integers(0, 1500, size=(B, 188)).astype(np.int32)  # pages shared between sequences
    c = random_cache(1500, H, D, page, 8, 24)
    q = g.standard_normal((B, H, D)).astype(np.float16)
    y = host(awq.awq_kv_attention(dev(q), c, dev(table), dev(lengths)))
    sub = {k: v[:, heads] for k, v in host_cache(c).items()}
    ref, tol = attend_ref(q[:, heads], sub, table, lengths, D ** -0.5, 8, 24)
    assert np.all(np.abs(y[:, heads] - ref) <= tol)
    assert np.all(y[3] == 0)


def test_attention_captured_while_lengths_move_on():
    """One captured call over a table for 20000 tokens, replayed for lengths that change how the
    work is shared out, with eager calls between: each replay is the eager result."""
    B, H, r, D = 5, 2, 4, 128
    g = np.random.default_rng(25)
    c = random_cache(1300, H, D, 16, 4, 26)
    tab = dev(g.integers(0, 1300, size=(B, 1250)).astype(np.int32))
    q = dev(g.standard_normal((B, H * r, D)).astype(np.float16))
    lengths = torch.ones(B, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        awq.awq_kv_attention(q, c, tab, lengths)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = awq.awq_kv_attention(q, c, tab, lengths)
    for n in ([1, 1, 1, 1, 1], [20000, 0, 1, 128, 129], [0, 0, 0, 0, 0], [300, 4096, 4097, 12, 700], [19000, 20000, 18000, 17, 3]):
        lengths.copy_(dev(np.array(n, np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(out).view(np.uint16), host(awq.awq_kv_attention(q, c, tab, lengths)).view(np.uint16))
        ref, tol = attend_ref(host(q), host_cache(c), host(tab), n, D ** -0.5, 4, 160)
        assert np.all(np.abs(host(out) - ref) <= tol)


def test_attention_of_bad_pages():
    """Entries outside the cache count as absent; a sequence of nothing else gives 0."""
    g = np.random.default_rng(1)
    table = g.permutation(60).astype(np.int32)[:40].reshape(4, 10)
    table[0, [0, 3]] = [-1, 2 ** 31 - 1]
    table[1] = -2 ** 31
    table[2, 9] = 42   # first entry past the cache (4 * 10 + 2 pages)
    table[table > 41] = 5
    table[2, 9] = 42
    y, _ = check_attention(4, [160, 150, 155, 20], 2, 2, 128, 16, 8, seed=4, table=table)
    assert np.all(y[1] == 0)


def test_attention_one_page_shared_and_max_len():
    table = np.zeros((2, 8), np.int32)  # the same page again and again
    check_attention(2, [128, 100], 1, 4, 64, 16, 4, seed=5, table=table.copy())
    check_attention(2, [1000, 70], 2, 4, 128, 16, 4, seed=6, max_len=130)
    check_attention(2, [1000, 70], 2, 4, 128, 16, 4, seed=6, max_len=1)


@pytest.mark.parametrize("magnitude", [2.0 ** -13, 1e-2, 40.0])
def test_attention_value_magnitudes(magnitude):
    """Scales near the smallest and far larger ones: the weights are brought to fp16's range."""
    check_attention(2, [700, 40], 2, 4, 128, 16, 4, seed=7, magnitude=magnitude, q_gain=min(1.0, 1 / magnitude))


def test_attention_peaked_rising_and_zero_scores():
    """Scores that rise along the sequence (the running maximum moves often), a softmax of one
    token, equal scores, and a negative scale."""
    check_attention(1, [1500], 1, 8, 128, 16, 8, seed=9, scale=3.0)
    check_attention(1, [1500], 1, 8, 128, 16, 8, seed=9, scale=0.0)
    check_attention(1, [1500], 1, 8, 128, 16, 8, seed=9, scale=-0.5)
    B, n, D = 1, 640, 64
    c = random_cache(40, 1, D, 16, 8, 3)
    t = np.arange(n)
    c["k_params"][:, 0, :, 0] = dev((0.001 * (1 + t)).reshape(40, 16).astype(np.float16))
    c["v_params"][:, 0, :, 0] = dev((0.0005 * 1.02 ** (t % 600)).reshape(40, 16).astype(np.float16))
    c["k_params"][:, 0, :, 1] = 0
    q = np.full((B, 2, D), 0.02, np.float16)
    q[0, 1] = -0.02
    table, lengths = np.arange(40, dtype=np.int32)[None], np.array([n], np.int32)
    y = host(awq.awq_kv_attention(dev(q), c, dev(table), dev(lengths), scale=1.0))
    ref, tol = attend_ref(q, host_cache(c), table, lengths, 1.0, 8, 8)
    assert np.all(np.abs(y - ref) <= tol)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("gain", [-22, -14, -8, 9])
def test_attention_query_magnitudes(gain, bits):
    """Queries from fp16's smallest numbers to its largest, with a scale that brings the scores back,
    and heads of mixed magnitudes: q enters as it is given."""
    check_attention(2, [700, 40], 2, 4, 128, 16, bits, seed=13, q_gain=2.0 ** gain, scale=2.0 ** (-gain - 3))
    g = np.random.default_rng(14)
    c = random_cache(20, 1, 64, 16, bits, 15)
    q = (g.standard_normal((1, 5, 64)) * np.exp2(np.array([-24, -10, 0, 4, 13])[None, :, None])).astype(np.float16)
    q[0, 1, 9] = 3.0
    q[0, 0] = 0
    table, lengths = np.arange(20, dtype=np.int32)[None], np.array([300], np.int32)
    y = host(awq.awq_kv_attention(dev(q), c, dev(table), dev(lengths), scale=2.0 ** -10))
    ref, tol = attend_ref(q, host_cache(c), table, lengths, 2.0 ** -10, bits, 4)
    assert np.all(np.abs(y - ref) <= tol)


@pytest.mark.parametrize("bits", [4, 8])
def test_attention_has_no_bias_over_long_sequences(bits):
    """The output of 100000 tokens of no common direction is a small difference of large sums: the
    mean error over the channels (in which roundings of the output cancel, as 5 standard
    deviations of their mean allow) stays within what the weights' 2^-22 and the products' 2^-22
    of those sums leave."""
    n, D, r = 100000, 128, 5
    c = random_cache(n // 16 + 1, 1, D, 16, bits, 29)
    q = np.random.default_rng(30).standard_normal((1, r, D)).astype(np.float16)
    table, lengths = np.random.default_rng(31).permutation(n // 16 + 1)[None].astype(np.int32), np.array([n], np.int32)
    y = host(awq.awq_kv_attention(dev(q), c, dev(table), dev(lengths))).astype(np.float64)
    h = host_cache(c)
    pg, at = table[0, np.arange(n) // 16], np.arange(n) % 16
    kc, vc = (unpack(h[x + "_codes"][pg, 0, at], bits).astype(np.float64) for x in "kv")
    kp, vp = (h[x + "_params"][pg, 0, at].astype(np.float64) for x in "kv")
    s = D ** -0.5 * (q[0].astype(np.float64) @ ((kc - kp[:, 1:]) * kp[:, :1]).T)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    out, mag = p @ ((vc - vp[:, 1:]) * vp[:, :1]), p @ ((vc + vp[:, 1:]) * vp[:, :1])
    err = (y[0] - out).reshape(r, D // 8, 8)
    rounding = 2.0 ** -11 * np.sqrt((out ** 2).mean())  # at most half a step each
    for i in range(8):
        e = err[:, :, i]
        assert abs(e.mean()) <= 2.0 ** -21 * mag.mean() + 5 * rounding / np.sqrt(3 * e.size)


@pytest.mark.parametrize("n", [40, 5000])
def test_attention_of_nan(n):
    """A NaN in one query head makes that head's output NaN, in one chunk and in many, and no other."""
    c = random_cache(320, 1, 64, 16, 4, 11)
    q = np.random.default_rng(12).standard_normal((1, 3, 64)).astype(np.float16)
    q[0, 1, 7] = np.nan
    table, lengths = np.arange(320, dtype=np.int32)[None], np.array([n], np.int32)
    y = host(awq.awq_kv_attention(dev(q), c, dev(table), dev(lengths)))
    assert np.isnan(y[0, 1]).all()
    q[0, 1, 7] = 0
    ref, tol = attend_ref(q, host_cache(c), table, lengths, 64 ** -0.5, 4, 40)
    assert np.all(np.abs(y - ref)[:, [0, 2]] <= tol[:, [0, 2]])


def test_attention_past_32_bit_offsets():
    """A cache whose halves pass 2^32 bytes and 2^31 words: first and last pages."""
    free, _ = torch.cuda.mem_get_info()
    if free < 30 << 30:
        pytest.skip("needs 30 GB of device memory")
    pages, H, D, page = (1 << 31) // (8 * 16 * 16) + 64, 8, 128, 16  # codes: 2^31 words and more
    c = awq.empty_kv_cache(pages, H, D, page=page, bits=4, device=DEV)
    assert c["k_codes"].numel() > 1 << 31
    g = np.random.default_rng(2)
    n = 40
    table = np.array([[pages - 1, 0, pages - 3]], np.int32)
    k, v = (g.standard_normal((n, H, D)).astype(np.float16) for _ in range(2))
    t = np.arange(n)
    slots = (table[0, t // page].astype(np.int64) * page + t % page).astype(np.int32)
    awq.awq_kv_write(dev(k), dev(v), dev(slots), c)
    kr, vr = awq.awq_kv_read(c, dev(slots), D)
    codes, scale, zero = quantise(k, 4)
    assert np.array_equal(host(kr), ((codes - zero[..., None]) * scale.astype(np.float64)[..., None]).astype(np.float16))
    q = g.standard_normal((1, 16, D)).astype(np.float16)
    y = host(awq.awq_kv_attention(dev(q), c, dev(table), dev(np.array([n], np.int32))))
    sub = {x: host(c[x][torch.tensor([pages - 1, 0, pages - 3], device=DEV)]) for x in c if x != "bits"}
    ref, tol = attend_ref(q, sub, np.array([[0, 1, 2]], np.int32), [n], D ** -0.5, 4, 1)
    assert np.all(np.abs(y - ref) <= tol)


@pytest.mark.parametrize("bits", [4, 8])
def test_decoding_step_together(bits):
    """A decoding loop as it is used: the fused product of 4-bit weights, its keys and values
    written into the cache, attention over what was written; eager, and as a captured graph
    whose page table and lengths move on between replays."""
    from test_gpu_experts import inputs, layer
    B, Hq, H, D, page, K = 3, 8, 2, 64, 16, 256
    _, p, sc, z = layer(1, (Hq + 2 * H) * D, K, 4, 21)
    cache = awq.empty_kv_cache(30, H, D, page=page, bits=bits, device=DEV)
    for n in ("k_params", "v_params"):
        cache[n].fill_(float("nan"))  # an unwritten slot that is used shows
    table = np.random.default_rng(4).permutation(30)[:18].reshape(B, 6).astype(np.int32)
    x = torch.empty((B, K), dtype=torch.float16, device=DEV)
    tab, slots, lengths = dev(table), torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)

    def step():
        qkv = awq.awq_gemm(x, p[0], sc[0], z[0]).view(B, Hq + 2 * H, D)
        awq.awq_kv_write(qkv[:, Hq:Hq + H], qkv[:, Hq + H:], slots, cache)
        return awq.awq_kv_attention(qkv[:, :Hq], cache, tab, lengths), qkv

    def advance(i):
        x.copy_(dev(inputs(B, K, 100 + i)))
        n = np.array([i + 1, i // 2 + 1, 0], np.int32)   # the third sequence is padding
        s = np.array([table[0, i // page] * page + i % page, table[1, (i // 2) // page] * page + (i // 2) % page, -1])
        lengths.copy_(dev(n))
        slots.copy_(dev(s.astype(np.int32)))
        return n

    def check(out, qkv, n):
        ref, tol = attend_ref(host(qkv)[:, :Hq], host_cache(cache), table, n, D ** -0.5, bits, 1)
        y = host(out).astype(np.float64)
        assert np.all(np.abs(y - ref) <= tol) and np.all(y[2] == 0)

    for i in range(20):
        n = advance(i)
        check(*step(), n)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(20, 40):
        n = advance(i)
        graph.replay()
        check(*captured, n)


def test_calls_on_two_streams_at_once_and_given_workspaces():
    """Long attention and routing on two streams side by side, each call with a workspace of its
    own (allocated, or given and full of NaN): the results of the calls one after the other."""
    g = np.random.default_rng(18)
    c = random_cache(900, 2, 128, 16, 4, 19)
    cases = []
    for i in range(2):
        q = dev(g.standard_normal((2, 16, 128)).astype(np.float16))
        table = dev(g.permutation(900)[:800].reshape(2, 400).astype(np.int32))
        lengths = dev(g.integers(5000, 6400, size=2).astype(np.int32))
        logits = dev(g.standard_normal((700, 33)).astype(np.float32))
        cases.append((q, table, lengths, logits))

    def run(case, ws=None):
        q, table, lengths, logits = case
        y = awq.awq_kv_attention(q, c, table, lengths, workspace=ws)
        r = awq.awq_moe_route(logits, 5)
        return [y.view(torch.int16), r["experts"], r["weights"].view(torch.int32), r["offsets"], r["rows"], r["pos"]]

    alone = [[host(t) for t in run(case)] for case in cases]
    need = awq.awq_kv_attention_workspace_bytes(2, 16, 2, 128, 4, 6400)
    assert need > 0
    streams, got = [torch.cuda.Stream() for _ in cases], [[], []]
    given = [torch.full((need // 4,), float("nan"), device=DEV) for _ in cases]
    torch.cuda.synchronize()
    for turn in range(6):
        for i, (s, case) in enumerate(zip(streams, cases)):
            with torch.cuda.stream(s):
                got[i].append(run(case, given[i] if turn % 2 else None))
    torch.cuda.synchronize()
    for i in range(2):
        for result in got[i]:
            assert all(np.array_equal(host(t), a) for t, a in zip(result, alone[i]))
    with pytest.raises(awq.AwqError):
        run(cases[0], given[0][:need // 4 - 64])


def test_refusals_of_the_binding():
    c = awq.empty_kv_cache(4, 2, 64, device=DEV)
    x = torch.zeros(3, 2, 64, dtype=torch.float16, device=DEV)
    i = torch.zeros(3, dtype=torch.int32, device=DEV)
    for f in (lambda: awq.awq_kv_write(x, x[:2], i, c), lambda: awq.awq_kv_write(x[:, :1], x[:, :1], i, c),
              lambda: awq.awq_kv_write(x.transpose(1, 2), x, i, c), lambda: awq.awq_kv_write(x, x, i[:2], c),
              lambda: awq.awq_kv_read(c, i, 128), lambda: awq.awq_kv_read({**c, "bits": 3}, i, 64),
              lambda: awq.awq_kv_attention(x, c, i[:, None][:2], i), lambda: awq.awq_kv_attention(x[:, :1], c, i[:, None], i),
              lambda: awq.awq_kv_attention(x, c, i[:, None], i, max_len=-1)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: awq.awq_kv_write(x.float(), x, i, c), lambda: awq.awq_kv_write(x, x, i.long(), c),
              lambda: awq.awq_kv_attention(x, c, i[:, None].long(), i)):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(awq.AwqError):
        awq.awq_kv_write(x[:1].expand(3, 2, 64), x, i, c)  # every token the same memory: a stride of 0
    with pytest.raises(awq.AwqError, match="finite"):
        awq.awq_kv_attention(x, c, i[:, None].contiguous(), i, scale=float("nan"))
