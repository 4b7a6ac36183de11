"""The tensor-memory forms of the attention when a bounded wait runs out, without a GPU fault: the copying warp gives up at the
third tile of each share, with earlier copies on their way (with an e4m3 cache the first product's warp does).  The call completes, the flag is set, no request is counted that was
not finished, and the next call is right."""
import pytest
import torch

from tests._gpu import status
from tests.test_gpu_paged_attention_shares import BF, E4, many_lengths, shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,Hq,W", [(BF, 4, 1), (BF, 8, 1), (BF, 12, 1), (BF, 12, 2), (E4, 12, 2), (BF, 13, 10), (E4, 13, 10)])
def test_every_role_leaves(cuda, kind, Hq, W):
    p = shared(kind, Hq, W, 64, many_lengths()).run(cuda)
    want, lse = p.out.clone(), p.lse.clone()
    cuda.kda_set_test_fault(cuda.KDA_TEST_FAULT_STALL_CACHE_COPIES)
    try:
        p.run(cuda)
    finally:
        cuda.kda_set_test_fault(cuda.KDA_TEST_FAULT_NONE)
    torch.cuda.synchronize()  # the kernels returned
    flags, rows = status(p.st)
    assert flags == cuda.KDA_DEV_TIMEOUT and rows < 64 * W * Hq
    p.run(cuda)
    assert status(p.st) == (0, 64 * W * Hq)
    assert torch.equal(p.out, want) and torch.equal(p.lse, lse)
