"""Workspace sizes of the operators around a projection (no GPU)."""
import os

import pytest

from qlora_parameter_efficient_amd import block, lq

pytestmark = pytest.mark.skipif(not os.path.exists(lq.LIB_PATH),
                                reason="liblq.so not built (run __graft_entry__.build())")


@pytest.mark.parametrize("V", [1, 3, 63, 64, 65, 200, 1000, 50257, 1 << 20])
def test_head_holds_one_piece_of_logits(V):
    """At most 2^28 logits, padding to 64 columns included, as float32 and bf16 (or 256
    rows of them), and 2^21 rows, which a launch of 1024 threads a row takes; partial
    sums of dH are at most 2^20 rows of K here."""
    size = block.lib().lq_head_loss_workspace
    K = 64
    M = min((1 << 25) - 1, (1 << 31) // K - 1)
    ld = -(-V // 64) * 64
    logits = min(max(1 << 28, 256 * ld), (1 << 21) * ld)
    assert 0 < size(M, V, K, 1, 0) <= 4 * logits + 4096
    assert size(M, V, K, 1, 1) <= 6 * logits + 4 * (1 << 21) + 4 * (1 << 20) * K + 4096


def rows_up_to(most):
    """Row counts whose neighbours have other tiles, splits and pieces."""
    edges = [1, 16, 17, 63, 64, 65, 128, 129, 256, 511, 767, 768, 769, 1024, 1025, 1535, 1536, 1537, 4096, 4097, 8128,
             8129, 8192, 8193, 16384, 16385, 65536, 65537, 262143]
    return sorted({m for m in edges + list(range(1, 9000, 37)) if m <= most})


def grows(size, most=1 << 20):
    last = 0
    for M in rows_up_to(most):
        now = size(M)
        assert now >= last, (M, now, last)
        last = now


@pytest.mark.parametrize("K", [64, 1024, 1025, 4096, 5000, 8192, 16384, 30000, 65536])
def test_norm_workspace_is_enough_for_fewer_rows(K):
    grows(lambda M: block.lib().lq_rmsnorm_bwd_workspace(M, K))


@pytest.mark.parametrize("op", [block.LQ_ADAPTERS_OP_FWD, block.LQ_ADAPTERS_OP_BWD])
@pytest.mark.parametrize("N,K,r,slots", [(4096, 4096, 64, 16), (11008, 4096, 32, 64), (4096, 11008, 11, 1), (64, 8128, 16, 300),
                                         (64, 64, 1, 4096), (1024, 1024, 7, 8)])
def test_adapter_workspace_is_enough_for_fewer_rows(op, N, K, r, slots):
    grows(lambda M: block.lib().lq_adapters_workspace_size(op, M, N, K, r, slots), ((1 << 31) - 1) // max(N, K))


@pytest.mark.parametrize("need_dh", [0, 1])
@pytest.mark.parametrize("V,K", [(32000, 4096), (50257, 2048), (128256, 4096), (1000, 512), (3, 64), (1 << 20, 1024), (9999, 16384)])
def test_head_workspace_is_enough_for_fewer_rows(V, K, need_dh):
    grows(lambda M: block.lib().lq_head_loss_workspace(M, V, K, 1, need_dh), ((1 << 31) - 1) // K)
