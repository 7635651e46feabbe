"""lq_adapters_bwd on pools whose gradients pass 2^32 elements."""
import pytest
import torch

from qlora_parameter_efficient_amd import block

from .gpu_helpers import DEV, announce

pytestmark = pytest.mark.gpu


def test_no_rows_clear_a_large_pools_gradients():
    """1025 places x 64 x 65536: dA has 2^32 + 2^22 elements, more than a launch has
    threads.  M = 0 writes zeros to all of it."""
    slots, r, N, K = 1025, 64, 64, 65536
    announce("gradients of 2^32 elements, no rows")
    q = block.AdapterPool(torch.empty((slots, r, K), dtype=torch.bfloat16, device=DEV),
                          torch.empty((slots, N, r), dtype=torch.bfloat16, device=DEV), torch.ones(slots, device=DEV))
    dA = torch.full((slots, r, K), 3.0, device=DEV)
    dB = torch.full((slots, N, r), 3.0, device=DEV)
    none = lambda c: torch.empty((0, c), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    block.lq_adapters_bwd(none(N), none(K), q, torch.empty(0, dtype=torch.int32, device=DEV), dA=dA, dB=dB)
    for part in list(dA.view(-1).split(1 << 28)) + [dB]:
        assert not bool(part.any())
