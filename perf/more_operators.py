"""The block norm, the 8-bit product and the token choice as measured work: their cases, inputs, plain
forms and 64-bit definitions.

Three operators of a decoder that stand around its packed layers, experts and cache:

* the norm between two blocks (``awq_norm``): the block's output is normed, gated, scaled and added to
  the residual stream, and the next block's input is normed from that, as fp16 or as rows of 8 bits;
* the product in 8-bit integers with a scale for each token and each channel (``awq_gemm_i8``), its
  rows quantised on the way, or handed over by the norm;
* the choice of the next token (``awq_sample``): temperature, top-k, top-p and min-p, from given random
  numbers.

``run`` computes the plain form (elementary torch operations in 32 bits, in 64 where a rounding or a
border decides) unless ``own`` is set, in which case it makes the framework's calls.  Sizes are those
of this repository's layers (4096, 11008, 8192, 28672) or generic ones.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # One decoding step of a small batch: residual sum and the next norm, latency is all there is.
        _norm("norm_step", T=4, N=4096),
        # A batch of images or utterances under conditioning: layer norms, each sequence with its own gate,
        # the residual stream kept in 32 bits; odd token count.
        _norm("norm_conditioned", T=2047, N=1408, layer=True, bias=True, gate="rows", wide=True),
        # A long prompt between two blocks with norms on both sides, gated, residuals scaled.
        _norm("norm_prompt", T=16384, N=8192, post=True, gate="channel", scale=0.22),
        # The norm that hands 8-bit rows to the product, for a decoding batch and for a prompt.
        dict(name="block_step", kind="block", T=24, K=4096, N=4096),
        dict(name="block_prompt", kind="block", T=4000, K=4096, N=11008),
        # One token through a wide layer: the weights are read once.
        dict(name="product_token", kind="product", M=1, K=4096, N=11008, scaled=False, wide=False),
        # A decoding batch through the long-row layer, rows divided by the layer's input scales.
        dict(name="product_batch", kind="product", M=77, K=11008, N=4096, scaled=True, wide=False),
        # The vocabulary's product of a batch, its logits in 32 bits; odd channel count.
        dict(name="product_logits", kind="product", M=32, K=4096, N=50021, scaled=False, wide=True),
        # A prompt through the widest layer: compute-bound.
        dict(name="product_prompt", kind="product", M=8192, K=8192, N=28672, scaled=False, wide=False),
        # One sequence's next token, all filters on.
        dict(name="sample_one", kind="sample", B=1, V=32000, half=False, filters="all", pad=0),
        # A serving batch, each row with its own settings (some greedy, some without a filter); rows of a
        # padded vocabulary.
        dict(name="sample_batch", kind="sample", B=61, V=50021, half=True, filters="mixed", pad=27),
        # A large batch over a large vocabulary.
        dict(name="sample_large", kind="sample", B=512, V=131072, half=True, filters="all", pad=0),
    ]


def _norm(name, **given):
    c = dict(kind="norm", T=1, N=8, layer=False, bias=False, post=False, residual=True, gate="none", scale=1.0, wide=False)
    c.update(given)
    if name is not None:
        c["name"] = name
    return c


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "norm", "block", "product", "product", "product", "sample", "sample", "sample"])
    if kind == "norm":
        N = 8 * _log(rng, 16, 2048)
        layer, residual = rng.random() < 0.3, rng.random() < 0.8
        return _norm(None, T=min(_log(rng, 1, 16384), 2 ** 26 // N), N=N, layer=layer,
                     bias=layer and rng.random() < 0.7, residual=residual, post=residual and rng.random() < 0.5,
                     gate=rng.choice(["none", "channel", "rows"]) if residual else "none",
                     scale=rng.choice([1.0, 0.22, 0.5]) if residual else 1.0, wide=rng.random() < 0.3)
    if kind in ("block", "product"):
        K, N, M = 128 * _log(rng, 2, 128), _log(rng, 32, 28672), _log(rng, 1, 8192)
        while M * N * K > 2 ** 40:
            M //= 2
        if kind == "block":
            return dict(kind=kind, T=M, K=K, N=N)
        return dict(kind=kind, M=M, K=K, N=N, scaled=rng.random() < 0.3, wide=rng.random() < 0.2)
    V = _log(rng, 300, 152000)
    return dict(kind=kind, B=min(_log(rng, 1, 512), 2 ** 26 // V), V=V, half=rng.random() < 0.5,
                filters=rng.choice(["none", "k", "p", "all", "mixed", "mixed"]), pad=rng.choice([0, 0, 1, 11, 64]))


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV)


def _rows(g, T, N):
    """Activations: a token's size varies, and some channels are outliers."""
    gain = torch.where(_uniform(g, N) < 0.005, 12.0, 1.0) * torch.exp(0.3 * _normal(g, N))
    return _normal(g, T, N) * gain * torch.exp(0.3 * _normal(g, T, 1))


def _weight_codes(g, N, K):
    """Rows of 8-bit weights as quantising bell-shaped rows leaves them, and their scales."""
    codes = torch.empty(N, K, dtype=torch.int8, device=DEV)
    step = max(1, 2 ** 26 // K)
    for a in range(0, N, step):
        b = min(N, a + step)
        codes[a:b] = torch.round(30 * _normal(g, b - a, K)).clamp(-127, 127).to(torch.int8)
    return codes, 0.02 / 30 * torch.exp(0.2 * _normal(g, N))


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    if c["kind"] in ("norm", "block"):
        T, N = c["T"], c["N"] if c["kind"] == "norm" else c["K"]
        h = 3 * _rows(g, T, N)
        st = dict(c, h=h if c.get("wide") else h.half(), weight=(1 + 0.2 * _normal(g, N)).half(),
                  y=_rows(g, T, N).half())
        if c["kind"] == "block":
            st["codes"], st["scales"] = _weight_codes(g, c["N"], N)
            return st
        rows = max(1, min(T, 16))  # sequences of a batch
        st["y"] = st["y"] if c["residual"] else None
        st["norm_bias"] = (0.1 * _normal(g, N)).half() if c["bias"] else None
        st["post_weight"] = (1 + 0.2 * _normal(g, N)).half() if c["post"] else None
        st["post_bias"] = (0.1 * _normal(g, N)).half() if c["post"] and c["bias"] else None
        st["gates"] = {"none": None, "channel": (0.5 * _normal(g, N)).half(),
                       "rows": (0.5 * _normal(g, rows, N)).half()}[c["gate"]]
        st["gate_rows"] = (torch.sort(torch.randint(0, rows, (T,), generator=g, device=DEV)).values.to(torch.int32)
                           if c["gate"] == "rows" else None)
        return st
    if c["kind"] == "product":
        codes, scales = _weight_codes(g, c["N"], c["K"])
        return dict(c, x=_rows(g, c["M"], c["K"]).half(), codes=codes, scales=scales,
                    s=torch.exp(0.4 * _normal(g, c["K"])) if c["scaled"] else None)
    B, V = c["B"], c["V"]
    # a few likely tokens over a broad background
    logits = 2.0 * _normal(g, B, V + c["pad"])
    logits += torch.where(_uniform(g, B, V + c["pad"]) < 30 / V, 6 * _uniform(g, B, V + c["pad"]) + 3, 0.0)
    st = dict(c, logits=(logits.half() if c["half"] else logits)[:, :V], u=_uniform(g, B))
    pick = lambda values: torch.tensor(values, device=DEV)[torch.randint(0, len(values), (B,), generator=g, device=DEV)]  # noqa: E731
    if c["filters"] == "mixed":
        st.update(temperature=pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.3]), top_k=pick([0, 0, 1, 20, 50, 400]).to(torch.int32),
                  top_p=pick([1.0, 1.0, 0.95, 0.9, 0.5]), min_p=pick([0.0, 0.0, 0.05, 0.1]))
    else:
        f = c["filters"]
        st.update(temperature=0.8, top_k=50 if f in ("k", "all") else 0, top_p=0.9 if f in ("p", "all") else 1.0,
                  min_p=0.02 if f == "all" else 0.0)
    return st


# --------------------------------------------------------------------------------- the plain form
def _plain_norm(v, weight, bias, layer):
    if layer:
        v = v - v.mean(1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * weight.float()
    return v if bias is None else v + bias.float()


def _plain_residual(st):
    h, y = st["h"].float(), st["y"].float()
    if st.get("post_weight") is not None:
        y = _plain_norm(y, st["post_weight"], st["post_bias"], st["layer"])
    if st.get("gates") is not None:
        y = y * (st["gates"].float() if st["gate_rows"] is None else st["gates"].float()[st["gate_rows"].long()])
    return (h + y * st.get("scale", 1.0)).to(st["h"].dtype)


def _norm_case(st):
    h = st["h"] if st["y"] is None else _plain_residual(st)
    x = _plain_norm(h.float(), st["weight"], st["norm_bias"], st["layer"]).half()
    return [x] if st["y"] is None else [h, x]


def _plain_product(codes_x, scales_x, codes_w, scales_w):
    return torch.matmul(codes_x.float(), codes_w.float().t()) * scales_x[:, None] * scales_w


def _block_case(st):
    h = _plain_residual(st)
    # the norm's factor 1 / rms drops out of the codes, which are rounded from the products in 64 bits
    t = h.double() * st["weight"].double()
    top = t.abs().amax(1, keepdim=True)
    codes = torch.round(127 * t / top.clamp(min=1e-300))
    scale = torch.rsqrt((h.float() ** 2).mean(1) + EPS) * top[:, 0].float() / 127
    return [h, _plain_product(codes, scale, st["codes"], st["scales"]).half()]


def _product_case(st):
    x = st["x"].float()
    if st["s"] is not None:
        x = x / st["s"]
    top = x.abs().amax(1, keepdim=True)
    codes = torch.round(127 * x.double() / top.double().clamp(min=1e-300))
    y = _plain_product(codes, top[:, 0] / 127, st["codes"], st["scales"])
    return y if st["wide"] else y.half()


def _column(v):
    return v[:, None] if isinstance(v, torch.Tensor) else v


def _sample_case(st):
    x = st["logits"].float()
    V = x.shape[1]
    order = torch.sort(x, dim=1, descending=True, stable=True)  # the lower index first where logits are equal
    t = torch.as_tensor(_column(st["temperature"]), device=DEV, dtype=torch.float32).double()
    d = (order.values - order.values[:, :1]).double()
    rank = torch.arange(V, device=DEV)
    # temperature 0 is the largest logit alone
    w = torch.where(t > 0, torch.exp(d / torch.where(t > 0, t, 1.0)), (rank == 0).double())
    k = torch.as_tensor(_column(st["top_k"]), device=DEV)
    w = torch.where((k <= 0) | (rank < k), w, 0.0)
    p = torch.as_tensor(_column(st["top_p"]), device=DEV, dtype=torch.float32).double()
    upto = torch.cumsum(w, 1)
    w = torch.where((p >= 1) | (upto - w < p * upto[:, -1:]), w, 0.0)
    w = torch.where(w >= torch.as_tensor(_column(st["min_p"]), device=DEV, dtype=torch.float32).double(), w, 0.0)
    back = torch.zeros_like(w).scatter_(1, order.indices, w)
    upto = torch.cumsum(back, 1)
    total = upto[:, -1:]
    token = (upto <= st["u"].double()[:, None] * total).sum(1, keepdim=True).clamp(max=V - 1)
    return [token[:, 0].to(torch.int32), (back.gather(1, token) / total)[:, 0].float()]


# -------------------------------------------------------------------------------------- one pass
def run(st):
    kind = st["kind"]
    if not own:
        return {"norm": _norm_case, "block": _block_case, "product": _product_case, "sample": _sample_case}[kind](st)
    import weight_only_quantization_gemm_amd as awq
    if kind == "norm":
        r = awq.awq_norm(st["h"], st["weight"], y=st["y"], bias=st["norm_bias"], post_weight=st["post_weight"],
                         post_bias=st["post_bias"], gate=st["gates"], gate_rows=st["gate_rows"], scale=st["scale"],
                         kind="layer" if st["layer"] else "rms", eps=EPS)
        return [r["x"]] if st["y"] is None else [r["h"], r["x"]]
    if kind == "block":
        r = awq.awq_norm(st["h"], st["weight"], y=st["y"], eps=EPS, quantize=True)
        return [r["h"], awq.awq_gemm_i8(r["x"], st["codes"], st["scales"], x_scales=r["scales"])]
    if kind == "product":
        return awq.awq_gemm_i8(st["x"], st["codes"], st["scales"], s=st["s"],
                               dtype=torch.float32 if st["wide"] else torch.float16)
    r = awq.awq_sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                       min_p=st["min_p"])
    return [r["tokens"], r["probs"]]


def work(case):
    c = case
    if c["kind"] == "norm":
        T, N, b = c["T"], c["N"], 4 if c["wide"] else 2
        rows = max(1, min(T, 16)) if c["gate"] == "rows" else int(c["gate"] == "channel")
        vectors = 1 + c["bias"] + c["post"] * (1 + c["bias"]) + rows
        moved = T * N * (b + 2 + (b + 2 if c["residual"] else 0))
        return dict(bytes=moved + 2 * vectors * N + (4 * T if c["gate"] == "rows" else 0),
                    flops=T * N * (4 + 2 * c["layer"] + c["bias"] + (4 * c["post"] + 3 if c["residual"] else 0)))
    if c["kind"] == "block":
        T, K, N = c["T"], c["K"], c["N"]
        return dict(bytes=T * K * 6 + 2 * K + N * K + 4 * N + 2 * T * N, flops=2 * T * N * K)
    if c["kind"] == "product":
        M, K, N = c["M"], c["K"], c["N"]
        return dict(bytes=2 * M * K + (4 * K if c["scaled"] else 0) + N * K + 4 * N + (4 if c["wide"] else 2) * M * N,
                    flops=2 * M * N * K)
    B, V = c["B"], c["V"]
    return dict(bytes=B * V * (2 if c["half"] else 4) + B * (12 + (16 if c["filters"] == "mixed" else 0)), flops=4 * B * V)


# ------------------------------------------------------------------------ the definition in 64 bits
def _exact_norm(v, weight, bias, layer):
    n = v.shape[1]
    if layer:
        v = v - (v.sum(1) / n)[:, None]
    v = weight.to(v.dtype) * v / torch.sqrt((v ** 2).sum(1) / n + EPS)[:, None]
    return v + bias.to(v.dtype) if bias is not None else v


def _exact_residual(st):
    """The new residual stream before its rounding."""
    add = st["y"].to(torch.float64)
    if st.get("post_weight") is not None:
        add = _exact_norm(add, st["post_weight"], st["post_bias"], st["layer"])
    gates = st.get("gates")
    if gates is not None:
        gates = gates.to(torch.float64)
        add = add * (gates[st["gate_rows"].long()] if st["gate_rows"] is not None else gates)
    return st["h"].to(torch.float64) + st.get("scale", 1.0) * add


def _exact_codes(v):
    top = v.abs().max(1).values
    return torch.round(v * 127 / torch.where(top > 0, top, 1.0)[:, None]), top / 127


def _exact_product(codes, scale, st):
    out = torch.empty(codes.shape[0], st["codes"].shape[0], dtype=torch.float64, device=DEV)
    step = max(1, 2 ** 28 // codes.shape[1])
    for a in range(0, out.shape[1], step):
        w = st["codes"][a:a + step].to(torch.float64) * st["scales"][a:a + step, None].to(torch.float64)
        out[:, a:a + step] = codes @ w.t() * scale[:, None]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    kind, f64 = st["kind"], torch.float64
    if kind == "norm":
        if st["y"] is None:
            return [_exact_norm(st["h"].to(f64), st["weight"], st["norm_bias"], st["layer"])]
        h = _exact_residual(st)
        # the next norm reads the residual stream as it is kept
        return [h, _exact_norm(h.to(st["h"].dtype).to(f64), st["weight"], st["norm_bias"], st["layer"])]
    if kind == "block":
        h = _exact_residual(st)
        kept = h.half().to(f64)
        codes, scale = _exact_codes(kept * st["weight"].to(f64))
        return [h, _exact_product(codes, scale / torch.sqrt((kept ** 2).sum(1) / kept.shape[1] + EPS), st)]
    if kind == "product":
        x = st["x"].to(f64)
        if st["s"] is not None:
            x = x / st["s"].to(f64)
        return _exact_product(*_exact_codes(x), st)
    # sampling: each row by itself, as the settings say
    B, V = st["logits"].shape
    probs = torch.empty(B, dtype=f64, device=DEV)
    setting = lambda name: (st[name].tolist() if isinstance(st[name], torch.Tensor)  # noqa: E731
                            else [torch.tensor(st[name], dtype=torch.float32).item()] * B)
    settings = zip(setting("temperature"), setting("top_k"), setting("top_p"), setting("min_p"), st["u"].tolist())
    for b, (t, k, p, m, u) in enumerate(settings):
        x = st["logits"][b].to(f64)
        if t <= 0:
            probs[b] = 1.0
            continue
        value, index = torch.sort(x, descending=True, stable=True)
        weight = torch.exp((value - value[0]) / t)
        n = min(int(k), V) if k > 0 else V
        total = weight[:n].sum()
        before = torch.cat([weight.new_zeros(1), weight[:n].cumsum(0)[:-1]])
        kept = weight[:n] >= m
        if p < 1:
            kept &= before < p * total
        index, weight = index[:n][kept], weight[:n][kept]
        index, at = torch.sort(index)
        upto = weight[at].cumsum(0)
        chosen = int(torch.searchsorted(upto, (u * upto[-1]).reshape(1), right=True))
        probs[b] = weight[at][min(chosen, index.numel() - 1)] / upto[-1]
    return [None, probs]
