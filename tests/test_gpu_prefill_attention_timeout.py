"""The tensor-memory kernels of the prompt attention when a bounded wait runs out, without a GPU fault: the copying warp gives up at
the third tile that a CTA walks, with earlier copies on their way.  The calls complete, the flag is set, only finished rows are
counted, and the next calls are right."""
import pytest
import torch

from tests import _prompt as P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,d,softcap", [(4, 2, 128, 0.0), (3, 1, 128, 5.0), (2, 2, 64, 0.0), (6, 1, 32, 5.0)])
def test_every_role_leaves(cuda, Hq, Hkv, d, softcap):
    lengths = [900, 100, 2000]
    q, k, v, d_out = P.inputs(3000, Hq, Hkv, d, torch.bfloat16, 21)
    args = (q, k, v, P.cu(lengths), 2000)
    want = P.run(cuda, *args, d_out, softcap=softcap)
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    cuda.kda_set_test_fault(cuda.KDA_TEST_FAULT_STALL_PROMPT_COPIES)
    try:
        got = P.run(cuda, *args, softcap=softcap, dev_status=status)
        torch.cuda.synchronize()  # the kernels returned
        flags, rows = status.tolist()
        assert flags == cuda.KDA_DEV_TIMEOUT and 100 * Hq <= rows < 3000 * Hq
        done = torch.zeros(3000, dtype=torch.bool, device="cuda")
        for a, n in ((0, 128), (900, 100), (1000, 128)):
            done[a:a + n] = True
        assert torch.equal(got["out"][done], want["out"][done])
        untouched = (got["out"] == 7.0).all(-1)
        assert (untouched | (got["out"] == want["out"]).all(-1)).all()
        status.zero_()
        grads = [torch.full_like(want[n], 7.0) for n in ("dq", "dk", "dv")]
        ws = torch.empty(cuda.kda_prefill_attention_backward_workspace_size(3000, 3, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
        call = (d_out, q, k, v, want["out"], want["lse"], args[3], 2000, *grads, ws)
        cuda.kda_prefill_attention_backward(*call, softcap=softcap, dev_status=status)
        torch.cuda.synchronize()
        flags, rows = status.tolist()
        assert flags == cuda.KDA_DEV_TIMEOUT and 100 * Hq <= rows < 3000 * Hq
    finally:
        cuda.kda_set_test_fault(cuda.KDA_TEST_FAULT_NONE)
    status.zero_()
    cuda.kda_prefill_attention_backward(*call, softcap=softcap, dev_status=status)
    again = P.run(cuda, *args, softcap=softcap)
    assert status.tolist() == [0, 3000 * Hq]
    for n, x in zip(("dq", "dk", "dv"), grads):
        assert torch.equal(x, want[n]), n
    assert torch.equal(again["out"], want["out"])
