"""The expert and key-value cache entry points on the host: size queries, refusals before
anything is launched, the alignment check of every device pointer, and the cache kernels'
address arithmetic (no GPU needed)."""
import os
import subprocess

import pytest
import torch

import weight_only_quantization_gemm_amd as awq
from weight_only_quantization_gemm_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, MISALIGNED, WS_SMALL = 1, 2, 3
FAKE, FAKE_MISALIGNED = 0x10000, 0x10008  # never dereferenced: the checks fail first

# A valid call of each entry point (by parameter), and its device pointers.
CALLS = {
    "awq_moe_plan": dict(experts=FAKE, T=5, E=8, top_k=2, offsets=FAKE, rows=FAKE, pos=FAKE, workspace=FAKE,
                         workspace_bytes=1 << 20, stream=None),
    "awq_moe_route": dict(logits=FAKE, logit_bytes=2, T=5, E=8, top_k=2, renormalize=1, experts=FAKE, weights=FAKE,
                          offsets=FAKE, rows=FAKE, pos=FAKE, workspace=FAKE, workspace_bytes=1 << 20, stream=None),
    "awq_gemm_grouped": dict(x=FAKE, x_rows=5, rows=FAKE, top_k=2, offsets=FAKE, s=FAKE, packed=FAKE, scales=FAKE,
                             zeros=FAKE, y=FAKE, R=10, E=8, N=64, K=256, group=128, bits=4, workspace=FAKE,
                             workspace_bytes=1 << 20, stream=None),
    "awq_moe_combine": dict(y=FAKE, R=10, pos=FAKE, weights=FAKE, T=5, top_k=2, N=64, out=FAKE, stream=None),
    "awq_kv_write": dict(k=FAKE, v=FAKE, k_stride=512, v_stride=512, slots=FAKE, k_codes=FAKE, k_params=FAKE,
                         v_codes=FAKE, v_params=FAKE, T=3, H=2, D=128, pages=4, page=16, bits=4, stream=None),
    "awq_kv_read": dict(k_codes=FAKE, k_params=FAKE, v_codes=FAKE, v_params=FAKE, slots=FAKE, k=FAKE, v=FAKE, T=3, H=2,
                        D=128, pages=4, page=16, bits=4, stream=None),
    "awq_kv_attention": dict(q=FAKE, q_stride=1024, k_codes=FAKE, k_params=FAKE, v_codes=FAKE, v_params=FAKE,
                             page_table=FAKE, table_width=64, lengths=FAKE, out=FAKE, B=3, Hq=8, Hkv=2, D=128, pages=4,
                             page=16, bits=4, scale=0.1, max_len=0, workspace=FAKE, workspace_bytes=1 << 24,
                             stream=None),
}
OPTIONAL = {"awq_gemm_grouped": {"rows", "s"}}


def call(entry, **changes):
    return getattr(_lib.load(), entry)(*dict(CALLS[entry], **changes).values())


def pointers(entry):
    return [k for k, v in CALLS[entry].items() if v == FAKE]


@pytest.mark.parametrize("entry", sorted(CALLS))
def test_every_pointer_is_checked(entry):
    for name in pointers(entry):
        assert call(entry, **{name: FAKE_MISALIGNED}) == MISALIGNED, name
        assert awq.awq_last_error() == f"{name} must be 16-byte aligned"
        if name not in OPTIONAL.get(entry, ()):
            assert call(entry, **{name: None}) == INVALID, name
            assert "NULL" in awq.awq_last_error()


BAD = {
    "awq_moe_plan": [dict(T=0), dict(E=0), dict(E=1025), dict(top_k=0), dict(top_k=65), dict(T=(1 << 24) + 1),
                     dict(T=1 << 23, top_k=3)],
    "awq_moe_route": [dict(T=0), dict(E=0), dict(E=1025), dict(top_k=9), dict(top_k=0), dict(logit_bytes=8),
                      dict(renormalize=2)],
    "awq_gemm_grouped": [dict(R=0), dict(x_rows=0), dict(x_rows=9, rows=None), dict(top_k=0), dict(E=0), dict(E=1025),
                         dict(N=0), dict(K=100), dict(group=64), dict(bits=8), dict(R=(1 << 24) + 1), dict(K=1 << 21), dict(K=(1 << 17) + 128),
                         dict(R=1 << 24, N=1 << 20, s=None), dict(R=1 << 24, s=FAKE),
                         dict(R=2048, E=1024, N=1 << 19, s=FAKE)],
    "awq_moe_combine": [dict(T=0), dict(R=0), dict(top_k=0), dict(N=12), dict(N=0), dict(T=1 << 24, N=1 << 20)],
    "awq_kv_write": [dict(T=0), dict(T=(1 << 22) + 1), dict(T=1 << 22, H=64, k_stride=8192, v_stride=8192), dict(H=0), dict(H=1025), dict(D=96), dict(page=24), dict(page=8),
                     dict(page=2048), dict(pages=0), dict(pages=1 << 27), dict(bits=3), dict(k_stride=128),
                     dict(v_stride=260)],
    "awq_kv_read": [dict(T=0), dict(D=32), dict(page=0), dict(pages=-1), dict(bits=16)],
    "awq_kv_attention": [dict(B=0), dict(B=65536), dict(Hq=7), dict(Hq=1), dict(Hkv=0), dict(D=80), dict(page=17),
                         dict(bits=2), dict(q_stride=1023), dict(q_stride=512), dict(table_width=0), dict(max_len=-1),
                         dict(table_width=1 << 26), dict(table_width=1 << 27), dict(scale=float("nan")),
                         dict(scale=float("inf")), dict(scale=2e19), dict(scale=-2e19)],
}


@pytest.mark.parametrize("entry,bad", [(e, b) for e in sorted(BAD) for b in BAD[e]], ids=str)
def test_bad_sizes_are_refused(entry, bad):
    assert call(entry, **bad) == INVALID
    assert awq.awq_last_error() != "no error"


def test_workspaces():
    lib = _lib.load()
    for entry, need in (("awq_moe_plan", awq.awq_moe_workspace_bytes(5, 8, 2)),
                        ("awq_moe_route", awq.awq_moe_workspace_bytes(5, 8, 2)),
                        ("awq_gemm_grouped", awq.awq_gemm_grouped_workspace_bytes(10, 256, True)),
                        ("awq_kv_attention", awq.awq_kv_attention_workspace_bytes(3, 8, 2, 128, 4, 1024))):
        assert need > 0 and need % 256 == 0
        assert call(entry, workspace_bytes=need - 1) == WS_SMALL
    assert awq.awq_gemm_grouped_workspace_bytes(10, 256, True) == 10 * 256 * 4
    assert awq.awq_gemm_grouped_workspace_bytes(2049, 256, True) == 2049 * 256 * 2
    assert awq.awq_gemm_grouped_workspace_bytes(10, 256, False) == 0
    assert awq.awq_gemm_grouped_workspace_bytes(10, 100, True) == 0
    assert awq.awq_moe_workspace_bytes(0, 8, 2) == 0 and awq.awq_moe_workspace_bytes(5, 8, 65) == 0
    assert awq.awq_kv_attention_workspace_bytes(1, 8, 8, 128, 4, 16) == 0  # one chunk: nothing to join
    assert awq.awq_kv_attention_workspace_bytes(1, 8, 3, 128, 4, 1000) == 0
    assert awq.awq_kv_attention_workspace_bytes(1, 8, 8, 128, 3, 1000) == 0
    assert awq.awq_kv_attention_workspace_bytes(1, 8, 8, 96, 4, 1000) == 0
    assert lib.awq_kv_codes_bytes(4, 2, 16, 128, 4) == 4 * 2 * 16 * 64
    assert lib.awq_kv_codes_bytes(4, 2, 16, 128, 8) == 4 * 2 * 16 * 128
    assert lib.awq_kv_params_bytes(4, 2, 16) == 4 * 2 * 16 * 4
    assert lib.awq_kv_codes_bytes(4, 2, 15, 128, 4) == 0 and lib.awq_kv_params_bytes(0, 2, 16) == 0


@pytest.mark.parametrize("R,E,N,K,bits,kernel", [
    (2, 8, 11008, 4096, 4, "grouped_ring_kernel<4,2,2> block=256 grid=688"),      # one token, two choices
    (8, 8, 64, 128, 3, "grouped_ring_kernel<3,2,2> block=64 grid=16"),            # one group: one wave
    (270, 64, 2048, 1408, 3, "grouped_ring_kernel<3,4,2> block=128 grid=2432"),
    (640, 64, 2048, 2048, 4, "grouped_ring_kernel<4,4,2> block=64 grid=3200"),    # ten rows an expert
    (641, 64, 2048, 2048, 4, "grouped_pipe_kernel<4,2,1,3> block=256 grid=640"),
    (320, 8, 4096, 11008, 4, "grouped_ring_kernel<4,4,2> block=128 grid=1728"),   # too few column tiles for the pipeline
    (321, 8, 4096, 11008, 4, "grouped_pipe_kernel<4,2,1,3> block=256 grid=256"),
    (3071, 8, 11008, 4096, 3, "grouped_pipe_kernel<3,2,1,3> block=256 grid=2432"),
    (12000, 8, 11008, 4096, 4, "grouped_pipe_kernel<4,4,2,3> block=512 grid=2432"),
    (12000, 8, 1000, 11008, 3, "grouped_pipe_kernel<3,4,2,2> block=512 grid=256"),  # long rows: two stages
    (12000, 8, 1000, 20480, 4, "grouped_pipe_kernel<4,2,1,3> block=256 grid=896"),  # no 256-row stages left
    (12000, 8, 1000, 24576, 4, "grouped_pipe_kernel<4,2,1,2> block=256 grid=896"),
    (12000, 8, 1000, 65536, 4, "grouped_ring_kernel<4,4,2> block=64 grid=12112"),
    (12000, 8, 1000, 131072, 4, "grouped_ring_kernel<4,2,2> block=64 grid=24224"),
    (1 << 24, 64, 32768 - 256, 4096, 4, "grouped_pipe_kernel<4,4,2,3> block=512 grid=8331136"),
])
def test_grouped_dispatch(R, E, N, K, bits, kernel):
    assert awq.awq_gemm_grouped_kernel(R, E, N, K, bits=bits) == kernel


def test_grouped_dispatch_refuses_what_the_product_refuses():
    for kw in (dict(R=0), dict(E=0), dict(N=0), dict(K=100), dict(bits=5), dict(R=1 << 24, N=1 << 20), dict(K=1 << 18)):
        with pytest.raises(awq.AwqError):
            awq.awq_gemm_grouped_kernel(**{**dict(R=10, E=8, N=64, K=256, bits=4), **kw})


def test_cache_buffers_have_the_documented_sizes():
    lib = _lib.load()
    for bits in awq.KV_BITS:
        for D in awq.KV_HEAD_DIMS:
            c = awq.empty_kv_cache(5, 3, D, page=32, bits=bits, device="cpu")
            assert c["k_codes"].numel() * 4 == lib.awq_kv_codes_bytes(5, 3, 32, D, bits)
            assert c["v_params"].numel() * 2 == lib.awq_kv_params_bytes(5, 3, 32)
    for bad in (dict(bits=3), dict(head_dim=96), dict(page=20), dict(page=8)):
        with pytest.raises(ValueError):
            awq.empty_kv_cache(**{**dict(pages=2, heads=1, head_dim=64, device="cpu"), **bad})


def test_binding_refuses_cpu_tensors_and_bad_shapes():
    f16, i32 = torch.float16, torch.int32
    cache = awq.empty_kv_cache(2, 1, 64, device="cpu")
    x = torch.zeros(2, 1, 64, dtype=f16)
    one = torch.zeros(2, dtype=i32)
    for f in (lambda: awq.awq_kv_write(x, x, one, cache), lambda: awq.awq_kv_read(cache, one, 64),
              lambda: awq.awq_kv_attention(x, cache, one[:, None], one), lambda: awq.awq_moe_plan(one[:, None], 4),
              lambda: awq.awq_moe_route(torch.zeros(2, 4), 2),
              lambda: awq.awq_moe_combine(x[:, 0], one, torch.zeros(2, 1)),
              lambda: awq.awq_gemm_grouped(torch.zeros(1, 128, dtype=f16), torch.zeros(1, 8, 16, dtype=i32),
                                           torch.zeros(1, 8, 1, dtype=f16), torch.zeros(1, 8, 1, dtype=torch.uint8),
                                           one)):
        with pytest.raises(ValueError, match="GPU"):
            f()


def test_cache_addresses_stay_inside(tmp_path):
    """Every row the kernels form from slots, page-table entries (bad ones among them) and
    lengths lies in the cache: the kernels' own arithmetic, compiled for the host."""
    exe = tmp_path / "kv_index_check"
    csrc = os.path.join(ROOT, "weight_only_quantization_gemm_amd", "csrc")
    subprocess.run(["g++", "-O1", "-Wall", "-Werror", "-I", csrc, os.path.join(ROOT, "tests", "kv_index_check.cpp"),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


def test_attention_split_covers_every_token_once(tmp_path):
    """The pieces attention's work is cut into by the lengths: the kernels' own arithmetic,
    compiled for the host."""
    exe = tmp_path / "kv_split_check"
    csrc = os.path.join(ROOT, "weight_only_quantization_gemm_amd", "csrc")
    subprocess.run(["g++", "-O1", "-Wall", "-Werror", "-I", csrc, os.path.join(ROOT, "tests", "kv_split_check.cpp"),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
