"""The largest batches of the grouped product that its header states: served just below each limit and
refused at it (host-only: the dispatch query, and refusals before anything is launched)."""
import pytest

import weight_only_quantization_gemm_amd as awq
from test_serve_abi import FAKE, INVALID, call

# kernel, rows of a tile, columns of a tile, limit, and batches that it serves (R, E, K)
LIMITS = [
    ("grouped_pipe_kernel<4,4,2,", 256, 256, 39, [(393216, 1024, 4096), (2400, 5, 4096), (1 << 24, 64, 4096)]),
    ("grouped_pipe_kernel<4,2,1,", 64, 256, 38, [(262144, 1024, 4096), (2400, 8, 4096)]),
    ("grouped_ring_kernel<4,4,2>", 16, 64, 33, [(2400, 1024, 4096), (20000, 8, 65536)]),
    ("grouped_ring_kernel<4,2,2>", 16, 32, 32, [(700, 1024, 4096), (20000, 8, 131072)]),
]


def widest(R, E, BM, BN, limit):
    """The largest N, in whole tiles, with N (R + (BM - 1) min(E, R)) below 2^limit."""
    rows = (R + (BM - 1) * min(E, R)) // BM  # row tiles
    return (2 ** limit // (BM * BN) - 1 - (127 if BM > 16 else 0)) // rows * BN


@pytest.mark.parametrize("kernel,BM,BN,limit,batches", LIMITS, ids=[c[0] for c in LIMITS])
def test_both_sides_of_the_largest_batch(kernel, BM, BN, limit, batches):
    for R, E, K in batches:
        N = widest(R, E, BM, BN, limit)
        # within a thousandth of the statement, or within a tile of it
        assert N * (R + (BM - 1) * min(E, R)) > 0.999 * 2 ** limit - 2 * BN * (R + (BM - 1) * min(E, R))
        assert awq.awq_gemm_grouped_kernel(R, E, N, K).startswith(kernel)
        with pytest.raises(awq.AwqError, match="refuses"):
            awq.awq_gemm_grouped_kernel(R, E, N + 2 * BN, K)


def test_two_numbers_of_a_scaled_input_halve_the_rows_of_a_tile():
    for R, E, BN, K in ((2048, 1024, 64, 256), (2048, 512, 32, 131072)):
        N = 2 ** (31 if BN == 32 else 32) // (R + 7 * min(E, R)) // BN * BN + 2 * BN
        assert awq.awq_gemm_grouped_kernel(R, E, N, K)  # without s it is served
        assert call("awq_gemm_grouped", R=R, E=E, N=N, K=K, s=FAKE, x_rows=R, workspace_bytes=1 << 40) == INVALID
        assert "exceed one launch" in awq.awq_last_error()
