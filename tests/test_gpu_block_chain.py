"""The block norm, the 8-bit product and the token choice as a decoding step uses them, with the cache
and the packed layers between, and the product against the layer it stands for."""
import numpy as np
import pytest
import torch

import weight_only_quantization_gemm_amd as awq
from test_gpu_sample import choose

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _half(g, *shape, scale=1.0):
    return torch.from_numpy((scale * g.standard_normal(shape)).astype(np.float16)).to(DEV)


class Model:
    """One attention block and the vocabulary's product: hidden 512, 4 query and 2 key-value heads of 128."""

    D, HQ, HKV, HID, VOCAB = 128, 4, 2, 512, 3001

    def __init__(self, seed):
        g = np.random.default_rng(seed)
        self.norms = [1 + 0.1 * _half(g, self.HID) for _ in range(3)]
        self.gate = _half(g, self.HID)
        self.qkv = awq.awq_pack_i8(_half(g, (self.HQ + 2 * self.HKV) * self.D, self.HID, scale=0.05))
        w = _half(g, self.HID, self.HQ * self.D, scale=0.05)
        r = awq.awq_quantize(w, _half(g, 64, self.HQ * self.D), awq.default_alpha_grid(4))
        self.o = (r["packed"], r["scales"], r["zeros"], r["s"])
        self.head = awq.awq_pack_i8(_half(g, self.VOCAB, self.HID, scale=0.1))

    def step(self, h, cache, slots, table, lengths, u):
        """One decoding step: the new residual stream, the logits, the tokens."""
        n = awq.awq_norm(h, self.norms[0], quantize=True)
        qkv = awq.awq_gemm_i8(n["x"], *self.qkv, x_scales=n["scales"]).view(len(h), -1, self.D)
        awq.awq_kv_write(qkv[:, self.HQ:self.HQ + self.HKV], qkv[:, self.HQ + self.HKV:], slots, cache)
        a = awq.awq_kv_attention(qkv[:, :self.HQ], cache, table, lengths).view(len(h), -1)
        p, sc, z, s = self.o
        y = awq.awq_gemm_scaled(a, s, p, sc, z)
        n = awq.awq_norm(h, self.norms[1], y=y, post_weight=self.norms[2], gate=self.gate, scale=0.5, quantize=True)
        logits = awq.awq_gemm_i8(n["x"], *self.head, x_scales=n["scales"], dtype=torch.float32)
        t = awq.awq_sample(logits, u, temperature=0.8, top_k=40, top_p=0.95, min_p=0.01)
        return n["h"], logits, t["tokens"], t["probs"], y, n


def _serve(B, seed):
    g = np.random.default_rng(seed)
    cache = awq.empty_kv_cache(pages=2 * B, heads=Model.HKV, head_dim=Model.D, page=16, bits=8, device=DEV)
    table = torch.arange(2 * B, dtype=torch.int32, device=DEV).view(B, 2).contiguous()
    return cache, table, _half(g, B, Model.HID), torch.from_numpy(g.random((8, B)).astype(np.float32)).to(DEV)


@pytest.mark.parametrize("B", [1, 5, 40])
def test_a_decoding_step_and_its_graph(B):
    """Eight steps: the tokens are the host's choice from the logits, the residual stream and the 8-bit
    rows are the formulas' of the step's own inputs; captured into a graph, each replay equals the eager step."""
    model = Model(3)
    cache, table, h, u = _serve(B, B)
    cache2 = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in cache.items()}
    static = [torch.zeros_like(h), torch.zeros(B, dtype=torch.int32, device=DEV), torch.ones(B, dtype=torch.int32, device=DEV),
              torch.zeros(B, device=DEV)]
    static[0].copy_(h)
    model.step(static[0], cache2, static[1], table, static[2], static[3])  # sizes are settled before capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = model.step(static[0], cache2, static[1], table, static[2], static[3])
    for i in range(8):
        slots = (table[:, i // 16] * 16 + i % 16).to(torch.int32).contiguous()
        lengths = torch.full((B,), i + 1, dtype=torch.int32, device=DEV)
        ui = u[i].clone()  # aligned like every operand
        new_h, logits, tokens, probs, y, n = model.step(h, cache, slots, table, lengths, ui)
        for s, v in zip(static, (h, slots, lengths, ui)):
            s.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got[:4], (new_h, logits, tokens, probs)):
            assert torch.equal(a, b), i
        for b in range(B):
            token, prob = choose(logits[b].cpu().numpy(), 0.8, 40, 0.95, 0.01, u[i, b].item())
            assert tokens[b].item() == token and abs(probs[b].item() - prob) <= 2.0 ** -23 * prob
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        p = f(y) / np.sqrt((f(y) ** 2).mean(1, keepdims=True) + 1e-5) * f(model.norms[2])
        want = f(h) + 0.5 * f(model.gate) * p
        # 2^-11 of the rounding, 2^-17 of what is summed before it
        assert np.all(np.abs(f(new_h) - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -17 * (np.abs(f(h)) + np.abs(p)) + 2.0 ** -25)
        v = (new_h.float() * model.norms[1].float()).double()
        assert torch.equal(n["x"].double(), torch.round(127 * v / v.abs().amax(1, keepdim=True)))
        h = new_h


@pytest.mark.parametrize("M,N,K", [(3, 200, 512), (40, 515, 1408), (300, 700, 1024)])
@pytest.mark.parametrize("scaled", [False, True])
def test_product_stands_for_the_layer(M, N, K, scaled):
    """y against x W^T in 64 bits.  With v = x / s and w = W * s, steps a of a row of v and b of one of w, each
    value is off by at most half a step (and the 2^-24 of forming it): |y - x W^T| <= b/2 sum |v| + a/2 (sum |w|
    + K b/2), to a thousandth for the roundings, and 2^-11 of the result."""
    g = np.random.default_rng(M)
    x = (g.standard_normal((M, K)) * np.where(g.random(K) < 0.02, 20, 1)).astype(np.float16)
    W = (0.05 * g.standard_normal((N, K))).astype(np.float16)
    s = np.exp(0.5 * g.standard_normal(K)).astype(np.float32) if scaled else np.ones(K, np.float32)
    ds = torch.from_numpy(s).to(DEV) if scaled else None
    codes, scales = awq.awq_pack_i8(torch.from_numpy(W).to(DEV), ds)
    y = awq.awq_gemm_i8(torch.from_numpy(x).to(DEV), codes, scales, s=ds, dtype=torch.float32).double().cpu().numpy()
    v, w = x.astype(np.float64) / s, W.astype(np.float64) * s
    a, b = np.abs(v).max(1)[:, None] / 127, np.abs(w).max(1)[None] / 127
    bound = b / 2 * np.abs(v).sum(1)[:, None] + a / 2 * (np.abs(w).sum(1)[None] + K * b / 2)
    want = x.astype(np.float64) @ W.astype(np.float64).T
    assert np.all(np.abs(y - want) <= 1.001 * bound + 2.0 ** -11 * np.abs(want))


def test_two_streams_at_once():
    """The same calls on two streams at the same time, each with its own outputs and workspaces."""
    g = np.random.default_rng(1)
    x, W = _half(g, 77, 4096), _half(g, 1024, 4096, scale=0.05)
    codes, scales = awq.awq_pack_i8(W)
    h, y, w = _half(g, 300, 4096), _half(g, 300, 4096), _half(g, 4096)
    logits, u = 3 * _half(g, 64, 20011), torch.rand(64, device=DEV)

    def run():
        n = awq.awq_norm(h, w, y=y, post_weight=w)
        t = awq.awq_sample(logits, u, top_p=0.9)
        return [awq.awq_gemm_i8(x, codes, scales), n["h"], n["x"], t["tokens"], t["probs"]]

    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(run())
    torch.cuda.synchronize()
    for results in got:
        for r in results:
            assert all(torch.equal(a, b) for a, b in zip(r, want))
