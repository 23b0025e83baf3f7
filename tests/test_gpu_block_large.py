"""Operands and results past 2^31 elements and bytes, checked at their far ends."""
import pytest
import torch

import weight_only_quantization_gemm_amd as awq
from test_gpu_sample import choose

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _free():
    torch.cuda.empty_cache()


@pytest.mark.parametrize("wide", [False, True])
def test_norm(wide):
    T, N = (1 << 18) + 5, 8200  # 2.15e9 elements
    torch.manual_seed(1)
    h = torch.empty(T, N, dtype=torch.float32 if wide else torch.float16, device=DEV).normal_()
    y = torch.empty(T, N, dtype=torch.float16, device=DEV).normal_()
    w = torch.randn(N, device=DEV).half()
    r = awq.awq_norm(h, w, y=y, post_weight=w)
    for rows in (slice(0, 2), slice(T - 2, T)):
        one = awq.awq_norm(h[rows].contiguous(), w, y=y[rows].contiguous(), post_weight=w)
        assert torch.equal(r["h"][rows], one["h"]) and torch.equal(r["x"][rows], one["x"])
    del r
    r = awq.awq_norm(h, w, y=y, quantize=True, h_out=h if not wide else None)
    assert r["x"][T - 1].abs().max().item() == 127
    del r, h, y
    _free()


def test_product_of_many_tokens():
    M, N, K = 70001, 32768, 128  # 2.3e9 results
    torch.manual_seed(2)
    x = torch.randint(-127, 128, (M, K), dtype=torch.int8, device=DEV)
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device=DEV)
    ones_m, ones_n = torch.ones(M, device=DEV), torch.full((N,), 2.0 ** -10, device=DEV)
    y = awq.awq_gemm_i8(x, w, ones_n, x_scales=ones_m)
    for rows in (slice(0, 2), slice(M - 3, M)):
        want = (x[rows].double() @ w.double().t() * 2.0 ** -10).half()
        assert torch.equal(y[rows], want)
    del x, w, y
    _free()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_product_of_many_channels(M):
    N, K = (1 << 20) + 77, 2176  # 2.3e9 codes
    torch.manual_seed(3)
    x = torch.randint(-127, 128, (M, K), dtype=torch.int8, device=DEV)
    w = torch.empty(N, K, dtype=torch.int8, device=DEV).random_(-127, 128)
    y = awq.awq_gemm_i8(x, w, torch.ones(N, device=DEV), x_scales=torch.ones(M, device=DEV), dtype=torch.float32)
    for rows in (slice(0, 2), slice(N - 100, N)):
        assert torch.equal(y[:, rows].double(), x.double() @ w[rows].double().t())  # below 2^24 and exact, or rounded once
    del x, w, y
    _free()


def test_rows_in_8_bits():
    M, K = 262149, 8320  # 2.2e9 values
    x = torch.empty(M, K, dtype=torch.float16, device=DEV).normal_()
    codes, scales = awq.awq_quantize_rows(x)
    for rows in (slice(0, 2), slice(M - 2, M)):
        c, s = awq.awq_quantize_rows(x[rows].contiguous())
        assert torch.equal(codes[rows], c) and torch.equal(scales[rows], s)
    del x, codes
    _free()


def test_token_choice():
    B, V = 20011, 131072  # 2.6e9 logits
    logits = torch.empty(B, V, dtype=torch.float16, device=DEV).normal_()
    logits *= 3
    u = torch.rand(B, device=DEV)
    for f in (dict(top_k=20, top_p=0.9), dict(top_p=0.2)):
        r = awq.awq_sample(logits, u, **f)
        for b in (0, B - 2, B - 1):
            token, prob = choose(logits[b].cpu().numpy(), 1.0, f.get("top_k", 0), f["top_p"], 0.0, u[b].item())
            assert r["tokens"][b].item() == token and abs(r["probs"][b].item() - prob) <= 2.0 ** -23 * prob
    del logits
    _free()
