"""Page ids outside the cache, in all forms of the attention over it: each is flagged, and its tokens are seen by no query.
Bounds as in test_gpu_paged_attention.py."""
import pytest
import torch

from tests._gpu import status
from tests.test_gpu_paged_attention import BF, E4, F32, Problem

pytestmark = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1
# cache, Hq, Hkv, W, d, types: the tensor-memory form for few rows, the many-rows form, the register form
FORMS = [(BF, 4, 1, 2, 128, BF), (BF, 12, 1, 2, 128, BF), (E4, 12, 1, 2, 128, BF), (E4, 4, 1, 1, 128, BF),
         (BF, 4, 2, 1, 64, BF), (E4, 6, 2, 1, 64, F32)]


@pytest.mark.parametrize("kind,Hq,Hkv,W,d,dt", FORMS)
@pytest.mark.parametrize("bad", [-1, -2, -3, LOW, HIGH, None])
def test_each_is_flagged(cuda, kind, Hq, Hkv, W, d, dt, bad):
    p = Problem([290, 70], W, Hq, Hkv, d, 32, kind, dt, dt)
    p.table[0, 3] = p.pages if bad is None else bad
    p.run(cuda)
    assert status(p.st) == (cuda.KDA_DEV_PAGE_OOB, 2 * W * Hq)
    p.table_cpu = p.table.cpu().long().clamp(0, p.pages - 1)
    p.check(hidden=set(range(96, 128)), only=[0])
    p.check(only=[1])


@pytest.mark.parametrize("kind,Hq,Hkv,W,d,dt", FORMS)
@pytest.mark.parametrize("bad", [-1, -2, HIGH])
def test_none_but_bad_pages(cuda, kind, Hq, Hkv, W, d, dt, bad):
    p = Problem([40, 70], W, Hq, Hkv, d, 32, kind, dt, dt)
    p.table[0, :2] = bad
    p.run(cuda)
    assert status(p.st)[0] == cuda.KDA_DEV_PAGE_OOB
    assert not p.out[0].any() and (p.lse[0] == -float("inf")).all()
    p.check(only=[1])


def test_entries_past_a_request_are_not_looked_at(cuda):
    for kind, Hq, Hkv, W, d, dt in FORMS:
        p = Problem([33, 64], W, Hq, Hkv, d, 32, kind, dt, dt)
        p.table[:, 2:] = HIGH
        p.run(cuda).check()
        assert status(p.st)[0] == 0
