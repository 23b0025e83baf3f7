"""awq_norm against its formula in 64 bits.

Tolerances.  A rounding to fp16 is off by at most 2^-11 of the value (2^-25 among its subnormals), one
to fp32 by 2^-24.  A sum of N <= 65536 squares runs over at most 64 terms a thread, 6 steps in a wave
and 16 waves, so the statistics are within 90 roundings, 2^-17 of what their terms' magnitudes sum to;
the remaining steps of a value are fewer than ten.  So a value within terms of magnitude A is within
2^-17 A of the formula before its last rounding.  The new residual stream is checked first; the norm
of it is then checked on the stream as it was returned, whose rounding is the operator's own."""
import numpy as np
import pytest
import torch

import weight_only_quantization_gemm_amd as awq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SLACK = 2.0 ** -17


def normed(v, w, b, layer, eps):
    """The norm of v (float64 [T][N]), and the magnitude of the terms it is summed from."""
    size = np.abs(v)
    if layer:
        mean = v.mean(1, keepdims=True)
        size = size + np.abs(v).mean(1, keepdims=True)
        v = v - mean
    r = 1 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    # a cancelled variance carries the mean's error, so the size is also relative to the rms
    x, size = v * r * w, size * r * np.abs(w) + np.abs(v * r * w) * (1 + size.max(1, keepdims=True) * r if layer else 1)
    return (x, size) if b is None else (x + b, size + np.abs(b))


def close(got, want, size, dtype, what):
    half = {torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}[dtype]
    tol = half * np.abs(want) + SLACK * size + (2.0 ** -25 if dtype == torch.float16 else 0)
    bad = np.abs(got.double().cpu().numpy() - want) > tol * (1 + 1e-9)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3])


def make(T, N, seed, wide=False, post=False, bias=False, gate=None, y=True, offset=0.0):
    g = np.random.default_rng(seed)
    half = lambda *s: g.standard_normal(s).astype(np.float16)  # noqa: E731
    h = (2 * g.standard_normal((T, N)) * np.exp(g.standard_normal((T, 1))) + offset).astype(np.float32 if wide else np.float16)
    d = dict(h=h, weight=half(N), y=half(T, N) if y else None, bias=half(N) if bias else None,
             post_weight=half(N) if post else None, post_bias=half(N) if post and bias else None, gate=None, gate_rows=None)
    if gate == "channel":
        d["gate"] = half(N)
    elif gate == "tokens":
        d["gate"] = half(T, N)
    elif gate == "rows":
        d["gate"], d["gate_rows"] = half(3, N), g.integers(-1, 5, T).astype(np.int32)  # -1, 3 and 4 add nothing
    return d


def check(d, layer=False, scale=1.0, eps=1e-5, on_gpu=None, **more):
    """Runs the call on d (numpy arrays; on_gpu overrides tensors) and checks all it returns."""
    dev = {k: torch.from_numpy(v).to(DEV) for k, v in d.items() if v is not None}
    dev.update(on_gpu or {})
    kind = "layer" if layer else "rms"
    r = awq.awq_norm(kind=kind, scale=scale, eps=eps, **dev, **more)
    f = {k: (v.astype(np.float64) if v is not None and v.dtype != np.int32 else v) for k, v in d.items()}
    h = f["h"]
    if d["y"] is not None:
        p, size = (f["y"], np.abs(f["y"])) if d["post_weight"] is None else normed(f["y"], f["post_weight"], f["post_bias"], layer, eps)
        gate = 1.0
        if d["gate"] is not None:
            gate = f["gate"]
            if d["gate_rows"] is not None:
                rows = d["gate_rows"]
                gate = np.where(((rows >= 0) & (rows < len(gate)))[:, None], gate[np.clip(rows, 0, len(gate) - 1)], 0.0)
        scale32 = float(np.float32(scale))
        close(r["h"], h + scale32 * gate * p, np.abs(h) + np.abs(scale32 * gate) * size, dev["h"].dtype, "h")
        h = r["h"].double().cpu().numpy()
    else:
        assert "h" not in r
    if "weight" not in d or d["weight"] is None:
        assert "x" not in r
        return r
    if more.get("quantize"):
        v = (h.astype(np.float32) * d["weight"].astype(np.float32)).astype(np.float64)
        top = np.abs(v).max(1)
        want = np.rint(127 * v / np.where(top > 0, top, 1)[:, None])  # exact: see code_of
        assert np.array_equal(r["x"].cpu().numpy(), want.astype(np.int8))
        scales = top / 127 / np.where(top > 0, np.sqrt((h * h).mean(1) + eps), 1)  # a row of zeros: 0
        assert np.all(np.abs(r["scales"].cpu().numpy() - scales) <= SLACK * scales)
    else:
        x, size = normed(h, f["weight"], f["bias"], layer, eps)
        close(r["x"], x, size, torch.float16, "x")
    return r


SIZES = [(1, 8), (3, 64), (5, 512), (2, 520), (9, 1024), (3, 1032), (4, 1408), (2, 2048), (3, 2056), (4, 4096), (2, 4104),
         (3, 5632), (2, 8192), (3, 8200), (2, 11008), (1, 16384), (2, 16392), (1, 28672), (2, 32768), (1, 32776), (2, 65536)]


@pytest.mark.parametrize("T,N", SIZES)
@pytest.mark.parametrize("wide", [False, True])
def test_residual_and_norm(T, N, wide):
    check(make(T, N, seed=N + T, wide=wide))
    check(make(T, N, seed=N + T + 1, wide=wide, post=True, gate="channel"), scale=0.22)
    check(make(T, N, seed=N + T + 2, wide=wide, y=False))


@pytest.mark.parametrize("T,N", [(1, 8), (5, 72), (9, 1024), (4, 1408), (3, 4104), (2, 16392)])
@pytest.mark.parametrize("wide", [False, True])
def test_layer_norm_with_biases(T, N, wide):
    check(make(T, N, seed=N, wide=wide, post=True, bias=True, gate="rows"), layer=True, scale=-0.5)
    check(make(T, N, seed=N + 1, wide=wide, y=False, bias=True, offset=100.0), layer=True)  # a mean far from zero


@pytest.mark.parametrize("gate", ["channel", "tokens", "rows"])
@pytest.mark.parametrize("T,N", [(1, 16), (300, 136), (7, 2048), (40, 4096)])
def test_gates(T, N, gate):
    check(make(T, N, seed=T, gate=gate))
    check(make(T, N, seed=T + 1, gate=gate, post=True, bias=True))


@pytest.mark.parametrize("T,N", [(1, 128), (5, 512), (300, 1024), (6, 4096), (3, 11008), (2, 65536)])
@pytest.mark.parametrize("wide", [False, True])
def test_rows_in_8_bits(T, N, wide):
    check(make(T, N, seed=N, wide=wide), quantize=True)
    check(make(T, N, seed=N + 1, wide=wide, post=True, gate="channel"), quantize=True, scale=0.5)
    check(make(T, N, seed=N + 2, wide=wide, y=False), quantize=True)


def test_codes_at_halves_and_tiny_rows():
    """Products whose 127 v / max|v| is a half exactly (rounded to even), next to a half, and rows
    whose largest product is near the smallest normal number or below."""
    N = 1024
    h = np.zeros((5, N), np.float32)
    h[0, :255] = np.arange(255) / 2.0  # 127 v / 127: 0, 1/2, 1, ...
    h[0, 255] = -127.0
    h[1, :N - 1] = (np.arange(N - 1) + 0.5) * np.float32(0.12512)
    h[1, -1] = 127.0 * 0.12512 * 8
    h[2] = np.linspace(-1, 1, N) * 2.0 ** -126
    h[3] = np.linspace(-1, 1, N) * 2.0 ** -140
    d = dict(h=h, weight=np.ones(N, np.float16), y=None, bias=None, post_weight=None, post_bias=None, gate=None, gate_rows=None)
    r = awq.awq_norm(torch.from_numpy(h).to(DEV), torch.from_numpy(d["weight"]).to(DEV), quantize=True)
    v = h.astype(np.float64)
    top = np.abs(v).max(1)
    want = np.rint(127 * v / np.where(top > 0, top, 1)[:, None]).astype(np.int8)
    got = r["x"].cpu().numpy()
    assert np.array_equal(got[[0, 1, 4]], want[[0, 1, 4]])
    assert np.array_equal(got[2:4], want[2:4])
    assert r["scales"][4].item() == 0.0  # a row of zeros


def test_zero_rows_and_no_eps():
    N = 256
    d = make(4, N, seed=1)
    d["h"][1] = 0
    d["y"][1] = 0
    r = check(d)
    assert not r["x"][1].any()
    check(make(4, N, seed=2), eps=0.0)


def test_residual_only():
    check(dict(make(6, 2048, seed=3, post=True), weight=None))


@pytest.mark.parametrize("N", [128, 4096])
def test_strides_and_in_place(N):
    d = make(6, N, seed=5, post=True)
    wide_h = torch.zeros(6, N + 24, dtype=torch.float16, device=DEV)
    wide_y = torch.zeros(6, 3 * N, dtype=torch.float16, device=DEV)
    wide_h[:, 8:8 + N] = torch.from_numpy(d["h"]).to(DEV)
    wide_y[:, N:2 * N] = torch.from_numpy(d["y"]).to(DEV)
    r = check(d, on_gpu=dict(h=wide_h[:, 8:8 + N], y=wide_y[:, N:2 * N]))
    h = torch.from_numpy(d["h"]).to(DEV)
    r2 = awq.awq_norm(h, torch.from_numpy(d["weight"]).to(DEV), y=wide_y[:, N:2 * N],
                      post_weight=torch.from_numpy(d["post_weight"]).to(DEV), h_out=h)
    assert r2["h"] is h and torch.equal(h, r["h"]) and torch.equal(r2["x"], r["x"])


def test_many_rows_and_repeats_are_equal():
    """More rows than blocks run at once, each as if alone; a second call gives the same bits."""
    d = make(5000, 264, seed=8, post=True, gate="rows")
    r = check(d)
    again = check(d)
    assert torch.equal(r["x"], again["x"]) and torch.equal(r["h"], again["h"])
    d = make(3001, 4096, seed=9)
    r = check(d)
    one = check({k: (v[2999:3000] if k in ("h", "y") else v) for k, v in d.items()})
    assert torch.equal(one["x"][0], r["x"][2999])


def test_other_stream_and_graph():
    d = {k: torch.from_numpy(v).to(DEV) for k, v in make(8, 1024, seed=4, post=True).items() if v is not None}
    want = awq.awq_norm(**d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = awq.awq_norm(**d)
    side.synchronize()
    assert torch.equal(got["x"], want["x"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = awq.awq_norm(**d)
    for i in range(3):
        d["h"].copy_(want["h"])
        d["y"].mul_(0.5)
        expect = awq.awq_norm(**d)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got["x"], expect["x"]) and torch.equal(got["h"], expect["h"])


def test_refusals():
    d = {k: torch.from_numpy(v).to(DEV) for k, v in make(4, 64, seed=4).items() if v is not None}
    h, w, y = d["h"], d["weight"], d["y"]
    for bad in (lambda: awq.awq_norm(h), lambda: awq.awq_norm(h, w[:32]), lambda: awq.awq_norm(h, w, y=y[:3]),
                lambda: awq.awq_norm(h, w, y=y[:, :32]), lambda: awq.awq_norm(h, w, kind="batch"),
                lambda: awq.awq_norm(h, w, gate=w), lambda: awq.awq_norm(h, w, y=y, gate=h[:2]),
                lambda: awq.awq_norm(h, w, y=y, gate=h[:, :32].contiguous()),
                lambda: awq.awq_norm(h, w, h_out=h), lambda: awq.awq_norm(h, y=y, quantize=True),
                lambda: awq.awq_norm(h, w, kind="layer", quantize=True), lambda: awq.awq_norm(h, w, bias=w, quantize=True),
                lambda: awq.awq_norm(h[:, ::2], w[:32]), lambda: awq.awq_norm(h, w, y=y, h_out=h[:3])):
        with pytest.raises((ValueError, awq.AwqError)):
            bad()
    with pytest.raises(awq.AwqError, match="aligned"):
        awq.awq_norm(h[:, 4:60], w[:56])
    with pytest.raises(TypeError):
        awq.awq_norm(h, w.float())


def test_rows_in_8_bits_without_eps_and_not_finite():
    """A row of zeros has scale 0 also where 1 / rms is infinite; one with a NaN or an infinity gives NaN."""
    for N in (256, 4096, 16384):
        d = make(5, N, seed=N)
        d["h"][1] = d["y"][1] = 0
        r = check(d, eps=0.0, quantize=True)
        assert r["scales"][1].item() == 0.0 and not r["x"][1].any()
        want = {k: v.clone() for k, v in r.items()}
        d["h"][3, N // 2 + 3] = np.nan
        d["y"][4, N - 1] = np.inf
        dev = {k: torch.from_numpy(v).to(DEV) for k, v in d.items() if v is not None}
        r = awq.awq_norm(**dev, eps=0.0, quantize=True)
        assert r["scales"][3:].isnan().all()
        assert torch.equal(r["x"][:3], want["x"][:3]) and torch.equal(r["scales"][:3], want["scales"][:3])


@pytest.mark.parametrize("N", [11000, 24576, 40000, 65528])
@pytest.mark.parametrize("wide", [False, True])
def test_long_rows_with_everything(N, wide):
    check(make(5, N, seed=N, wide=wide, post=True, bias=True, gate="rows"), layer=True, scale=0.75)
    check(make(3, N, seed=N + 1, wide=wide, post=True, gate="tokens"), quantize=True)
    check(make(2, N, seed=N + 2, wide=wide, y=False, bias=True, offset=50.0), layer=True)
