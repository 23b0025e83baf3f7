"""The expert and key-value cache operators as measured work: their cases, inputs, plain forms and
64-bit definitions.

Three operators of a decoding step with low-bit weights, and what belongs to them:

* experts: the router (``awq_moe_route``), the products grouped by expert (``awq_gemm_grouped``) and
  the weighted sum of a token's experts (``awq_moe_combine``);
* the cache: keys and values quantised as they are written and read back (``awq_kv_write``,
  ``awq_kv_read``);
* attention of one new token of each sequence over that cache (``awq_kv_attention``).

``run`` computes the plain form (elementary torch operations in 32 bits) unless ``own`` is set, in
which case it makes the framework's calls.  Sizes are those of this repository's layers (4096, 11008,
8192) or generic ones.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 128


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # Router of a decoding step over a small batch: latency is all there is.
        dict(name="route_step", kind="route", T=32, E=64, k=6, half=True, renorm=True),
        # Router over a long prompt with many experts and fp32 logits.
        dict(name="route_prompt", kind="route", T=16384, E=128, k=8, half=False, renorm=False),
        # One token through two of eight wide experts: the gate matrix of each is read once.
        dict(name="experts_token", kind="experts", T=1, E=8, k=2, K=4096, N=11008, bits=4, gather=True, scaled=False),
        # A decoding batch over 64 narrow experts (most have a handful of rows, some none), 3-bit
        # codes, each expert with the input scales of its own quantisation; 11 groups a row.
        dict(name="experts_batch", kind="experts", T=45, E=64, k=6, K=1408, N=2048, bits=3, gather=True, scaled=True),
        # A prompt through eight wide experts: compute-bound, groups of about 1500 rows.
        dict(name="experts_prompt", kind="experts", T=6000, E=8, k=2, K=4096, N=11008, bits=4, gather=True,
             scaled=False),
        # The weighted sum for one decoding batch, and for a prompt.
        dict(name="combine_step", kind="combine", T=24, k=6, N=2048),
        dict(name="combine_prompt", kind="combine", T=8192, k=4, N=4096),
        # A decoding batch's new keys and values into a 4-bit cache, as slices of the fused product.
        dict(name="cache_step", kind="cache", T=64, Hq=32, H=8, D=128, page=16, bits=4),
        # A prompt's keys and values into an 8-bit cache, heads not grouped.
        dict(name="cache_prompt", kind="cache", T=8000, Hq=32, H=32, D=128, page=64, bits=8),
        # A single sequence of ordinary length: the split over the length is all the parallelism.
        dict(name="attend_single", kind="attend", B=1, L=2000, Hkv=8, ratio=4, D=128, page=16, bits=4),
        # A serving batch of ragged lengths over a 4-bit cache.
        dict(name="attend_batch", kind="attend", B=64, L=6000, Hkv=8, ratio=8, D=128, page=16, bits=4),
        # Two very long sequences over an 8-bit cache with small heads.
        dict(name="attend_long", kind="attend", B=2, L=150001, Hkv=8, ratio=5, D=64, page=64, bits=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["route", "experts", "experts", "combine", "cache", "attend", "attend"])
    if kind == "route":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256])
        return dict(kind=kind, T=_log(rng, 1, 8192), E=E, k=rng.randint(1, 8), half=rng.random() < 0.5,
                    renorm=rng.random() < 0.5)
    if kind == "experts":
        E = rng.choice([4, 8, 16, 32, 64])
        K = 128 * _log(rng, 4, 64)
        N = _log(rng, 256, 8192)
        k = rng.randint(1, min(8, E))
        if E * N * K > 2 ** 28.5:
            N = max(256, int(2 ** 28.5 / (E * K)))
        T = _log(rng, 1, 4096)
        while T * k * N * K > 2 ** 38:
            T = max(1, T // 2)
        return dict(kind=kind, T=T, E=E, k=k, K=K, N=N, bits=rng.choice([4, 4, 3]), gather=rng.random() < 0.7,
                    scaled=rng.random() < 0.3)
    if kind == "combine":
        return dict(kind=kind, T=_log(rng, 1, 8192), k=rng.randint(1, 8), N=8 * _log(rng, 64, 512))
    if kind == "cache":
        H = rng.choice([1, 2, 4, 8, 32])
        D = rng.choice([64, 128, 256])
        return dict(kind=kind, T=min(_log(rng, 1, 6000), 2 ** 24 // (H * D)), Hq=H * rng.choice([1, 4, 8]), H=H, D=D,
                    page=rng.choice([16, 32, 64]), bits=rng.choice([4, 8]))
    D, bits, Hkv = rng.choice([64, 128, 128, 256]), rng.choice([4, 4, 8]), rng.choice([1, 2, 4, 8, 32])
    tokens = 2 ** 28 // (Hkv * D)  # bounds the plain form's fp32 keys and values
    L = min(_log(rng, 1, 100000), tokens)
    most = tokens // L
    return dict(kind=kind, B=max(1, min(_log(rng, 1, 128), most)), L=L, Hkv=Hkv, ratio=rng.choice([1, 2, 4, 5, 8, 16]),
                D=D, page=rng.choice([16, 32, 64, 128]), bits=bits)


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _words(g, *shape):
    return torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)


def _pairs(g, T, E, k):
    """Router logits with some experts liked more than others, and their k largest."""
    logits = _normal(g, T, E) * 1.5 + _normal(g, E)
    return logits, logits.topk(k, dim=1).indices


def _sorted_pairs(experts, E):
    """Pairs (token, choice) in order of expert: group offsets, pair of each row, row of each pair."""
    flat = experts.reshape(-1)
    rows = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(rows)
    pos[rows] = torch.arange(rows.numel(), device=DEV)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    return offsets.to(torch.int32), rows.to(torch.int32), pos.to(torch.int32)


def _pool(g, pages, H, P, D, bits, wide):
    """One half of a cache, filled as by quantising bell-shaped rows (`wide`: with some outlier channels)."""
    words = torch.empty(pages, H, P, D * bits // 32, dtype=torch.int32, device=DEV)
    params = torch.empty(pages, H, P, 2, dtype=torch.float16, device=DEV)
    gain = torch.ones(H, 1, D, device=DEV)
    if wide:
        gain = torch.where(torch.rand(H, 1, D, generator=g, device=DEV) < 0.03, 4.0, gain)
    step = max(1, 2 ** 25 // (H * P * D))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        codes, scale, zero = _quantise(_normal(g, b - a, H, P, D) * gain, bits)
        words[a:b] = _pack_codes(codes, bits)
        params[a:b] = torch.cat([scale, zero], -1).to(torch.float16)
    return words, params


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    if c["kind"] == "route":
        logits, _ = _pairs(g, c["T"], c["E"], 1)
        return dict(c, logits=logits.half() if c["half"] else logits)
    if c["kind"] == "experts":
        T, E, k, K, N, bits = (c[n] for n in ("T", "E", "k", "K", "N", "bits"))
        G = K // GROUP
        offsets, rows, _ = _sorted_pairs(_pairs(g, T, E, k)[1], E)
        x = _normal(g, T if c["gather"] else T * k, K)
        x *= torch.where(torch.rand(K, generator=g, device=DEV) < 0.01, 20.0, 1.0)
        zeros = torch.randint(6, 10, (E, N, 2 * ((G + 1) // 2)), generator=g, device=DEV, dtype=torch.uint8)
        if bits == 3:
            zeros = zeros - 4 - zeros % 2  # 2 or 4
        if G % 2:
            zeros[..., -1] = 0
        return dict(c, x=x.half(), offsets=offsets, rows=rows if c["gather"] else None,
                    s=torch.exp(0.4 * _normal(g, E, K)) if c["scaled"] else None,
                    packed=_words(g, E, N, K // 8 if bits == 4 else 3 * (K // 32)),
                    scales=(0.02 / 2 ** (bits - 2) * torch.exp(0.2 * _normal(g, E, N, G))).half(),
                    zeros=zeros[..., 0::2] | (zeros[..., 1::2] << 4))
    if c["kind"] == "combine":
        T, k, N = c["T"], c["k"], c["N"]
        experts = _pairs(g, T, 64, k)[1]
        return dict(c, y=_normal(g, T * k, N).half(), pos=_sorted_pairs(experts, 64)[2],
                    weights=torch.softmax(_normal(g, T, k), 1))
    if c["kind"] == "cache":
        T, Hq, H, D, P, bits = (c[n] for n in ("T", "Hq", "H", "D", "page", "bits"))
        qkv = _normal(g, T, Hq + 2 * H, D).half()  # the fused product's output: k and v are slices of it
        pages = -(-T // P) + 8
        cache = dict(k_codes=_words(g, pages, H, P, D * bits // 32), v_codes=_words(g, pages, H, P, D * bits // 32),
                     k_params=torch.ones(pages, H, P, 2, dtype=torch.float16, device=DEV),
                     v_params=torch.ones(pages, H, P, 2, dtype=torch.float16, device=DEV), bits=bits)
        slots = torch.randperm(pages, generator=g, device=DEV)[:, None] * P + torch.arange(P, device=DEV)
        return dict(c, k_new=qkv[:, Hq:Hq + H], v_new=qkv[:, Hq + H:], cache=cache,
                    slots=slots.reshape(-1)[:T].to(torch.int32).contiguous())
    B, L, H, D, P, bits = (c[n] for n in ("B", "L", "Hkv", "D", "page", "bits"))
    width = -(-L // P)
    lengths = torch.tensor(_lengths(c), device=DEV, dtype=torch.int32)
    pages = B * width + 3
    k_codes, k_params = _pool(g, pages, H, P, D, bits, True)
    v_codes, v_params = _pool(g, pages, H, P, D, bits, False)
    table = torch.randperm(pages, generator=g, device=DEV)[:B * width].reshape(B, width).to(torch.int32).contiguous()
    return dict(c, q=_normal(g, B, H * c["ratio"], D).half(), table=table, lengths=lengths,
                cache=dict(k_codes=k_codes, k_params=k_params, v_codes=v_codes, v_params=v_params, bits=bits))


def _lengths(c):
    """Ragged lengths of a batch: from a third of the longest to the longest, the first being that."""
    B, L = c["B"], c["L"]
    return [max(1, L - (L * 2 // 3) * ((7 * b) % 16) // 15) for b in range(B)]


# --------------------------------------------------------------------------------- the plain form
# Channel order of the 4-bit word: nibble p holds channel (0, 2, 4, 6, 1, 3, 5, 7)[p].
_ORDER = (0, 4, 1, 5, 2, 6, 3, 7)  # nibble of channel i


def _unpack_codes(words, bits):
    """The codes (int32) of packed words [..., W]: [..., W * 32 / bits]."""
    if bits == 8:
        sh = torch.arange(0, 32, 8, device=words.device, dtype=torch.int32)
        return words[..., None].bitwise_right_shift(sh).bitwise_and(255).flatten(-2)
    if bits == 4:
        sh = 4 * torch.tensor(_ORDER, device=words.device, dtype=torch.int32)
        return words[..., None].bitwise_right_shift(sh).bitwise_and(15).flatten(-2)
    # three words of 32 channels: channel 2p + h in bits 3 (p % 5) + 16 h of word p / 5; the last
    # pair's bits b in bit 15 + 16 h of word b
    w = words.unflatten(-1, (-1, 3))
    p = torch.arange(30, device=words.device) // 2
    sh = (3 * (p % 5) + 16 * (torch.arange(30, device=words.device) % 2)).to(torch.int32)
    body = w[..., p // 5].bitwise_right_shift(sh).bitwise_and(7)
    place = torch.tensor([1, 2, 4], device=words.device, dtype=torch.int32)
    last = [(w.bitwise_right_shift(b).bitwise_and(1) * place).sum(-1, keepdim=True, dtype=torch.int32) for b in (15, 31)]
    return torch.cat([body] + last, -1).flatten(-2)


def _pack_codes(codes, bits):
    """The packed words (int32) of codes [..., D] held as any whole numbers."""
    n = 32 // bits
    c = codes.to(torch.int64).unflatten(-1, (-1, n))
    sh = bits * (torch.tensor(_ORDER, device=c.device) if bits == 4 else torch.arange(n, device=c.device))
    w = (c << sh).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _quantise(v, bits):
    """Codes, scale and zero point of each row of v [..., D] (fp32)."""
    top = float(2 ** bits - 1)
    lo, hi = v.amin(-1, keepdim=True).clamp(max=0), v.amax(-1, keepdim=True).clamp(min=0)
    scale = ((hi - lo) / top).clamp(min=2.0 ** -14).half().float()
    zero = torch.round(-lo / scale).clamp(0, top)
    return (torch.round(v / scale) + zero).clamp(0, top), scale, zero


def _weights(packed, scales, zeros, K, bits):
    """The dequantised weights, fp32 [E][N][K]."""
    G = K // GROUP
    z = torch.stack([zeros & 15, zeros >> 4], -1).flatten(-2)[..., :G].float()
    w = _unpack_codes(packed, bits).float().unflatten(-1, (G, GROUP))
    return ((w - z[..., None]) * scales.float()[..., None]).flatten(-2)


def _route(st):
    x, k, E = st["logits"].float(), st["k"], st["E"]
    # the stable order puts the lower index first where logits are equal
    order = torch.sort(x, dim=1, descending=True, stable=True)
    experts = order.indices[:, :k]
    w = torch.exp(order.values - order.values[:, :1])
    w = w[:, :k] / (w[:, :k] if st["renorm"] else w).sum(1, keepdim=True)
    offsets, rows, pos = _sorted_pairs(experts, E)
    return dict(experts=experts.to(torch.int32), weights=w, offsets=offsets, rows=rows, pos=pos)


def _grouped(st):
    x, offsets, K, bits = st["x"], st["offsets"].long(), st["K"], st["bits"]
    R, E = st["T"] * st["k"], st["E"]
    at = torch.arange(R, device=x.device)
    expert = torch.searchsorted(offsets, at, right=True) - 1
    xs = x[st["rows"].long() // st["k"]].float() if st["gather"] else x.float()
    if st["s"] is not None:
        xs = xs / st["s"][expert]
    if R <= E:  # few rows: each with the weights of its expert
        w = _weights(st["packed"][expert], st["scales"][expert], st["zeros"][expert], K, bits)
        return torch.bmm(w, xs[:, :, None])[:, :, 0].half()
    w = _weights(st["packed"], st["scales"], st["zeros"], K, bits)
    pad = torch.zeros(E, int((offsets[1:] - offsets[:-1]).max()), K, device=x.device)
    pad[expert, at - offsets[expert]] = xs
    return torch.bmm(pad, w.transpose(1, 2))[expert, at - offsets[expert]].half()


def _combine(st):
    y = st["y"][st["pos"].long()].float().unflatten(0, (st["T"], st["k"]))
    return (y * st["weights"][:, :, None]).sum(1).half()


def _cache(st):
    c, got = st["cache"], []
    for new, codes, params in ((st["k_new"], c["k_codes"], c["k_params"]), (st["v_new"], c["v_codes"], c["v_params"])):
        page, at = st["slots"].long() // st["page"], st["slots"].long() % st["page"]
        q, scale, zero = _quantise(new.float(), st["bits"])
        codes[page, :, at] = _pack_codes(q, st["bits"])
        params[page, :, at] = torch.cat([scale, zero], -1).half()
        back, p = _unpack_codes(codes[page, :, at], st["bits"]).float(), params[page, :, at].float()
        got.append(((back - p[..., 1:]) * p[..., :1]).half())
    return got


def _attend(st):
    q, c, table, D, H = st["q"].float(), st["cache"], st["table"].long(), st["D"], st["Hkv"]
    B = q.shape[0]

    def half(codes, params):  # [B][H][L][D]
        codes, params = codes[table].transpose(1, 2).flatten(2, 3), params[table].transpose(1, 2).flatten(2, 3).float()
        return (_unpack_codes(codes, st["bits"]).float() - params[..., 1:]) * params[..., :1]

    k = half(c["k_codes"], c["k_params"])
    s = torch.matmul(q.view(B, H, -1, D), k.transpose(2, 3)) * D ** -0.5
    del k
    gone = torch.arange(s.shape[-1], device=q.device) >= st["lengths"][:, None, None, None]
    p = torch.exp(s.masked_fill(gone, -math.inf) - s.masked_fill(gone, -math.inf).amax(-1, keepdim=True))
    out = torch.matmul(p / p.sum(-1, keepdim=True), half(c["v_codes"], c["v_params"]))
    return out.reshape(B, -1, D).half()


# -------------------------------------------------------------------------------------- one pass
def run(st):
    kind = st["kind"]
    if not own:
        return {"route": _route, "experts": _grouped, "combine": _combine, "cache": _cache, "attend": _attend}[kind](st)
    import weight_only_quantization_gemm_amd as awq
    if kind == "route":
        return awq.awq_moe_route(st["logits"], st["k"], renormalize=st["renorm"])
    if kind == "experts":
        return awq.awq_gemm_grouped(st["x"], st["packed"], st["scales"], st["zeros"], st["offsets"], rows=st["rows"],
                                    top_k=st["k"] if st["gather"] else 1, s=st["s"])
    if kind == "combine":
        return awq.awq_moe_combine(st["y"], st["pos"], st["weights"])
    if kind == "cache":
        awq.awq_kv_write(st["k_new"], st["v_new"], st["slots"], st["cache"])
        return list(awq.awq_kv_read(st["cache"], st["slots"], st["D"]))
    return awq.awq_kv_attention(st["q"], st["cache"], st["table"], st["lengths"])


def work(case):
    c = case
    if c["kind"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return dict(bytes=T * E * (2 if c["half"] else 4) + T * k * 16 + (E + 1) * 4, flops=4 * T * E)
    if c["kind"] == "experts":
        T, E, k, K, N, G = c["T"], c["E"], c["k"], c["K"], c["N"], c["K"] // GROUP
        active = E * (1 - (1 - k / E) ** T)  # experts expected to have a row
        weights = active * N * (K * c["bits"] / 8 + 2 * G + (G + 1) // 2)
        return dict(bytes=weights + (T if c["gather"] else T * k) * K * 2 + T * k * N * 2 + (T * k + E + 1) * 4 +
                    (active * K * 4 if c["scaled"] else 0), flops=2 * T * k * N * K)
    if c["kind"] == "combine":
        T, k, N = c["T"], c["k"], c["N"]
        return dict(bytes=T * k * N * 2 + T * N * 2 + T * k * 8, flops=2 * T * k * N)
    if c["kind"] == "cache":
        rows = 2 * c["T"] * c["H"]  # written, and read back
        return dict(bytes=rows * (4 * c["D"] + 2 * (c["D"] * c["bits"] // 8 + 4)) + 8 * c["T"], flops=10 * rows * c["D"])
    n, Hq, D = sum(_lengths(c)), c["Hkv"] * c["ratio"], c["D"]
    return dict(bytes=n * c["Hkv"] * 2 * (D * c["bits"] // 8 + 4) + c["B"] * Hq * D * 4, flops=4 * n * Hq * D)


# ------------------------------------------------------------------------ the definition in 64 bits
def _code_at(words, i, bits):
    """Code of channel i (a tensor of channel numbers) of packed rows, by the format's statement."""
    words = words.long() & 0xFFFFFFFF
    if bits == 3:
        w, q = i // 32, i % 32
        pair, upper = q // 2, (q % 2) * 16
        plain = words[..., 3 * w + (pair // 5).clamp(max=2)] >> (3 * (pair % 5) + upper) & 7
        odd = sum((words[..., 3 * w + b] >> (15 + upper) & 1) << b for b in range(3))
        return torch.where(pair < 15, plain, odd)
    if bits == 4:
        return words[..., i // 8] >> (4 * (4 * (i % 2) + i % 8 // 2)) & 15
    return words[..., i // 4] >> (8 * (i % 4)) & 255


def exact(case, seed):
    st = prepare(case, seed)
    kind, f64 = st["kind"], torch.float64
    if kind == "route":
        x = st["logits"].to(f64)
        e = torch.exp(x - x.amax(1, keepdim=True))
        # k times the largest left, the first of equal ones
        index = torch.arange(st["E"], device=DEV)
        w = []
        left = e.clone()
        for _ in range(st["k"]):
            best = torch.where(left == left.amax(1, keepdim=True), index, st["E"]).amin(1, keepdim=True)
            w.append(torch.gather(e, 1, best))
            left.scatter_(1, best, -1.0)
        w = torch.cat(w, 1)
        w = w / (w if st["renorm"] else e).sum(1, keepdim=True)
        return dict(experts=None, weights=w, offsets=None, rows=None, pos=None)
    if kind == "experts":
        K, bits, k = st["K"], st["bits"], st["k"]
        i = torch.arange(K, device=DEV)
        off = st["offsets"].tolist()
        out = torch.zeros(off[-1], st["N"], dtype=f64, device=DEV)
        for e in range(st["E"]):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            zero = st["zeros"][e].long()[:, i // GROUP // 2] >> (4 * (i // GROUP % 2)) & 15
            w = (_code_at(st["packed"][e], i, bits) - zero).to(f64) * st["scales"][e].to(f64)[:, i // GROUP]
            x = st["x"][a:b] if st["rows"] is None else st["x"][st["rows"][a:b].long() // k]
            x = x.to(f64)
            if st["s"] is not None:
                x = x / st["s"][e].to(f64)
            out[a:b] = x @ w.t()
        return out
    if kind == "combine":
        out = torch.zeros(st["T"], st["N"], dtype=f64, device=DEV)
        for j in range(st["k"]):
            out += st["weights"][:, j, None].to(f64) * st["y"][st["pos"].view(-1, st["k"])[:, j].long()].to(f64)
        return out
    if kind == "cache":
        got = []
        for new in (st["k_new"], st["v_new"]):
            v, top = new.to(f64), 2.0 ** st["bits"] - 1
            lo, hi = torch.minimum(v.amin(2), v.new_zeros(())), torch.maximum(v.amax(2), v.new_zeros(()))
            step = torch.maximum((hi - lo) / top, v.new_tensor(2.0 ** -14)).to(torch.float16).to(f64)[..., None]
            zero = torch.round(-lo[..., None] / step).clamp(0, top)
            got.append(((torch.round(v / step) + zero).clamp(0, top) - zero) * step)
        return got
    c, D, H, P, r = st["cache"], st["D"], st["Hkv"], st["page"], st["ratio"]
    i = torch.arange(D, device=DEV)
    out = torch.zeros(st["B"], H * r, D, dtype=f64, device=DEV)
    for b, n in enumerate(st["lengths"].tolist()):
        t = torch.arange(n, device=DEV)
        page, at = st["table"][b].long()[t // P], t % P
        for h in range(H):
            k, v = ((_code_at(c[x + "_codes"][page, h, at], i, st["bits"]) - c[x + "_params"][page, h, at, 1:].to(f64)) *
                    c[x + "_params"][page, h, at, :1].to(f64) for x in "kv")
            s = st["q"][b, h * r:(h + 1) * r].to(f64) @ k.t() / math.sqrt(D)
            out[b, h * r:(h + 1) * r] = torch.softmax(s, 1) @ v
    return out
