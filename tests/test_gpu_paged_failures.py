"""Waits of the paged attention kernels that run out: the kernel says so and
returns, with its copies landed and its products complete, and the next calls
are right.  Nothing here faults or hangs a GPU: a hook keeps the producers from
issuing copies, and every wait has a limit of a second."""
import time

import pytest
import torch

from paged_harness import PagedCase, assert_rows, reference_rows
from test_gpu_paged import context, run_attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def lose_copies(hd, orc, case, ctx, stage):
    """A call whose producers stop at `stage`, then the same call whole; a first call makes the set-up's time no matter."""
    d = case.device()
    rows = list(range(0, case.rows, 11)) + [case.rows - 1]
    want = reference_rows(orc, case, rows)
    assert_rows(want, *run_attn(hd, ctx, case, d))
    assert hd.hybrid_decode_device_errors(ctx) == 0
    hd.hybrid_decode_inject_lost_copy(ctx, stage)
    t0 = time.monotonic()
    try:
        run_attn(hd, ctx, case, d)
    finally:
        hd.hybrid_decode_inject_lost_copy(ctx, -1)
    assert time.monotonic() - t0 < 8, "waits of a second each, one after the other"
    assert hd.hybrid_decode_device_errors(ctx) == 8
    for _ in range(2):
        assert_rows(want, *run_attn(hd, ctx, case, d))
    assert hd.hybrid_decode_device_errors(ctx) == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("spans", [[(900, 70), (0, 200), (300, 33)], [(9000, 70), (5, 20)]], ids=["short", "cut"])
@pytest.mark.parametrize("stage", [0, 3, 6])
def test_chunks(hd, orc, kv, spans, stage):
    """Stage 3 leaves a block of two operands half loaded, stage 6 a ring that has gone round."""
    lose_copies(hd, orc, PagedCase(110 + stage, spans, kv=kv), context(hd, kv=kv), stage)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("stage", [0, 5, 14])
def test_single_tokens(hd, orc, kv, stage):
    """Stage 5 leaves the ring's last slot empty, stage 14 is in the second round of the barriers."""
    lose_copies(hd, orc, PagedCase(120 + stage, [(19000, 1), (300, 1), (9000, 1), (18000, 1)] * 2, kv=kv, single=True),
                context(hd, kv=kv), stage)
