"""The entry points around the layers (block norm, 8-bit rows and product, token choice) on the
host: size queries, refusals before anything is launched, and the alignment check of every device
pointer (no GPU needed)."""
import pytest
import torch

import weight_only_quantization_gemm_amd as awq
from weight_only_quantization_gemm_amd import _lib

INVALID, MISALIGNED, WS_SMALL = 1, 2, 3
FAKE, FAKE_MISALIGNED = 0x10000, 0x10008  # never dereferenced: the checks fail first

# A valid call of each entry point (by parameter), and its device pointers.
CALLS = {
    "awq_norm": dict(h=FAKE, h_bytes=2, h_stride=64, y=FAKE, y_stride=72, post_weight=FAKE, post_bias=FAKE, gate=FAKE,
                     gate_rows=FAKE, gates=2, scale=1.0, weight=FAKE, bias=FAKE, kind=1, eps=1e-5, h_out=FAKE, x=FAKE,
                     x_scales=None, T=5, N=64, stream=None),
    "awq_quantize_rows": dict(x=FAKE, x_stride=256, s=FAKE, M=5, K=256, codes=FAKE, scales=FAKE, stream=None),
    "awq_pack_i8": dict(W=FAKE, s=FAKE, N=5, K=256, codes=FAKE, scales=FAKE, stream=None),
    "awq_gemm_i8": dict(x=FAKE, x_scales=None, s=FAKE, codes=FAKE, scales=FAKE, y=FAKE, y_bytes=2, M=5, N=64, K=256,
                        workspace=FAKE, workspace_bytes=1 << 20, stream=None),
    "awq_sample": dict(logits=FAKE, logit_bytes=2, stride=100, B=5, V=100, temperature=FAKE, temperature_value=1.0,
                       top_k=FAKE, top_k_value=0, top_p=FAKE, top_p_value=1.0, min_p=FAKE, min_p_value=0.0, u=FAKE,
                       tokens=FAKE, probs=FAKE, stream=None),
}
# pointers that may be left out by themselves
OPTIONAL = {"awq_norm": {"post_bias", "gate_rows", "bias"}, "awq_quantize_rows": {"s"}, "awq_pack_i8": {"s"},
            "awq_gemm_i8": {"s", "workspace"}, "awq_sample": {"temperature", "top_k", "top_p", "min_p", "probs"}}


def call(entry, **changes):
    return getattr(_lib.load(), entry)(*dict(CALLS[entry], **changes).values())


@pytest.mark.parametrize("entry", sorted(CALLS))
def test_every_pointer_is_checked(entry):
    for name in [k for k, v in CALLS[entry].items() if v == FAKE]:
        assert call(entry, **{name: FAKE_MISALIGNED}) == MISALIGNED, name
        assert awq.awq_last_error() == f"{name} must be 16-byte aligned"
        if name not in OPTIONAL[entry]:
            assert call(entry, **{name: None}) == INVALID, name


def test_scales_of_quantised_rows_are_checked():
    assert call("awq_norm", kind=0, bias=None, x_scales=FAKE_MISALIGNED) == MISALIGNED
    assert call("awq_gemm_i8", s=None, x_scales=FAKE_MISALIGNED) == MISALIGNED


BAD = {
    "awq_norm": [dict(T=0), dict(T=(1 << 24) + 1), dict(N=0), dict(N=12), dict(N=65544, h_stride=65544, y_stride=65544),
                 dict(h_bytes=8), dict(kind=2), dict(kind=-1), dict(eps=-1e-6), dict(eps=float("nan")),
                 dict(eps=float("inf")), dict(scale=float("nan")), dict(scale=float("inf")), dict(h_stride=56),
                 dict(h_stride=68), dict(y_stride=0), dict(y_stride=66), dict(h_stride=1 << 31), dict(gates=0),
                 dict(gates=(1 << 24) + 1), dict(gate_rows=None),  # two gate rows for five tokens, and no rows named
                 dict(h_stride=128),               # h_out is h, whose rows are strided
                 dict(x_scales=FAKE),              # rows in 8 bits of a layer norm
                 dict(kind=0, x_scales=FAKE),      # ... or with a bias
                 dict(y=None, h_out=None),         # post_weight and gate of no y
                 dict(y=None, h_out=None, post_weight=None, post_bias=None, gate=None, gate_rows=None, weight=None,
                      bias=None, x=None),          # nothing to compute
                 dict(weight=None, x=None)],       # a bias of no weight
    "awq_quantize_rows": [dict(M=0), dict(M=(1 << 24) + 1), dict(K=0), dict(K=100), dict(K=(1 << 17) + 128, x_stride=1 << 18),
                          dict(x_stride=248), dict(x_stride=260)],
    "awq_pack_i8": [dict(N=0), dict(N=(1 << 24) + 1), dict(K=64), dict(K=(1 << 17) + 128)],
    "awq_gemm_i8": [dict(M=0), dict(M=(1 << 22) + 1), dict(N=0), dict(N=(1 << 24) + 1), dict(M=1 << 22, N=(1 << 14) + 1),
                    dict(K=0), dict(K=130), dict(K=(1 << 17) + 128), dict(y_bytes=1), dict(x_scales=FAKE)],
    "awq_sample": [dict(B=0), dict(B=(1 << 20) + 1), dict(V=0), dict(V=(1 << 20) + 1, stride=1 << 21), dict(stride=99),
                   dict(stride=1 << 39), dict(logit_bytes=1), dict(temperature_value=float("nan")),
                   dict(top_p_value=float("nan")), dict(min_p_value=float("nan"))],
}


@pytest.mark.parametrize("entry,bad", [(e, b) for e in sorted(BAD) for b in BAD[e]], ids=str)
def test_bad_arguments_are_refused(entry, bad):
    assert call(entry, **bad) == INVALID
    assert awq.awq_last_error() != "no error"


def test_workspaces():
    need = awq.awq_gemm_i8_workspace_bytes(500, 64, 256, False)
    assert need >= 500 * 256 + 4 * 500 and need % 256 == 0  # the rows' codes and scales
    assert call("awq_gemm_i8", M=500, workspace_bytes=need - 1) == WS_SMALL
    assert call("awq_gemm_i8", M=500, workspace=None, workspace_bytes=need) == INVALID
    assert awq.awq_gemm_i8_workspace_bytes(0, 64, 256, False) == 0
    assert awq.awq_gemm_i8_workspace_bytes(5, 64, 100, False) == 0


def test_wrappers_refuse_cpu_tensors_and_wrong_types():
    h = torch.zeros(2, 64, dtype=torch.float16)
    w = torch.zeros(64, dtype=torch.float16)
    for f in (lambda: awq.awq_norm(h, w), lambda: awq.awq_quantize_rows(h), lambda: awq.awq_pack_i8(h),
              lambda: awq.awq_gemm_i8(h, torch.zeros(3, 64, dtype=torch.int8), torch.zeros(3)),
              lambda: awq.awq_sample(h, torch.zeros(2))):
        with pytest.raises(ValueError, match="GPU tensor"):
            f()
    with pytest.raises(TypeError, match="float16 or torch.float32"):
        awq.awq_norm(h.double(), w)
    with pytest.raises(TypeError):
        awq.awq_sample(h.to(torch.bfloat16), torch.zeros(2))
    with pytest.raises(TypeError):
        awq.awq_quantize_rows(h.float())


@pytest.mark.parametrize("M,N,K,quantized,kernel", [
    (1, 11008, 4096, False, "gemm_i8_skinny_kernel<1,4,4,1> block=256 grid=688"),   # quantises its own row
    (1, 4096, 65536, False, "gemm_i8_kernel<32,128,1,4,4,64> block=256 grid=160 shares=5"),  # too long a row for that
    (1, 4096, 4096, True, "gemm_i8_skinny_kernel<1,8,4,0> block=512 grid=256"),
    (32, 4096, 4096, True, "gemm_i8_skinny_kernel<2,8,2,0> block=512 grid=256"),
    (64, 1408, 2048, True, "gemm_i8_skinny_kernel<4,8,2,0> block=512 grid=88"),
    (16, 11008, 4096, True, "gemm_i8_kernel<32,64,1,2,6,64> block=128 grid=172 shares=1"),
    (16, 50021, 4096, True, "gemm_i8_kernel<32,128,1,4,4,64> block=256 grid=391 shares=1"),  # a wide layer
    (64, 28672, 8192, True, "gemm_i8_kernel<64,64,1,2,5,64> block=128 grid=448 shares=1"),
    (77, 4096, 11008, True, "gemm_i8_kernel<128,128,2,4,4,64> block=512 grid=224 shares=7"),
    (500, 4096, 1024, True, "gemm_i8_kernel<64,128,1,4,3,64> block=256 grid=256 shares=1"),
    (128, 28672, 8192, True, "gemm_i8_kernel<128,128,2,4,4,64> block=512 grid=224 shares=1"),
    (8192, 28672, 8192, True, "gemm_i8_kernel<256,256,2,4,4,32> block=512 grid=3584 shares=1"),
])
def test_product_dispatch(M, N, K, quantized, kernel):
    assert awq.awq_gemm_i8_kernel(M, N, K, quantized) == kernel


def test_product_workspaces():
    """None for a quantised x without shares of K, nor for the one row a kernel quantises itself."""
    assert awq.awq_gemm_i8_workspace_bytes(8192, 28672, 8192, True) == 0
    assert awq.awq_gemm_i8_workspace_bytes(1, 11008, 4096, False) == 0
    assert awq.awq_gemm_i8_workspace_bytes(77, 4096, 11008, True) == 7 * 77 * 4096 * 4
    assert awq.awq_gemm_i8_workspace_bytes(8192, 28672, 8192, False) == 8192 * 8192 + 8192 * 4
