"""One workspace for window and score decodes of many sizes."""
import numpy as np
import pytest
import torch

from bounded_helpers import DEV, Cache
from test_gpu_bounded import check_scores, check_window, new_err, pkv, run_scores, run_window  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 4), ("f16", 64, 8), ("f32", 128, 2)])
def test_one_workspace_for_batches_of_all_sizes(pkv, dtype, D, G):
    """Batches of 16, 1, 8, 3 and 16 sequences that are split into pieces, both operators in turn, on a
    workspace of the largest: what each gives on a workspace of its own, and the exact values."""
    caches = {B: Cache([3000 - 17 * s for s in range(B)], 8, G, D, 16, dtype, seed=B) for B in (16, 1, 8, 3)}
    ws = pkv.new_scores_workspace(16, 8 * G, 8, D, 3000)
    assert ws.numel() >= pkv.decode_window_workspace_bytes(16, 8 * G, 8, D)
    err = new_err()
    for B in (16, 1, 16, 8, 3, 16, 1, 3, 8, 16):
        c = caches[B]
        out = run_window(pkv, c, 2900, 4, ws, err)
        check_window(c, out, 2900, 4, f"B={B}")
        assert torch.equal(out, run_window(pkv, c, 2900, 4))
        new = torch.full((B, 8, 3000), float("nan"), device=DEV)
        out = run_scores(pkv, c, None, new, ws, err)
        check_scores(c, out, None, new, f"B={B}")
        assert (ws[:pkv.WINDOW_COUNTER_BYTES] == 0).all()
    assert int(err.item()) == 0


def test_a_small_calls_workspace_for_a_larger_call(pkv):
    """Sizes below the least workspace have the same number of bytes: the workspace of one sequence
    passes for a batch."""
    few, many = Cache((2500,), 2, 4, 128, 16, "bf16"), Cache([2500] * 16, 2, 4, 128, 16, "bf16")
    need = pkv.decode_window_workspace_bytes(16, 8, 2, 128)
    del_me = torch.full((pkv.decode_scores_workspace_bytes(1, 8, 2, 128, 2500),), 0xFF, dtype=torch.uint8, device=DEV)
    del del_me  # what the allocator hands out next
    ws = pkv.new_scores_workspace(1, 8, 2, 128, 2500)
    assert ws.numel() >= need
    ws[pkv.WINDOW_COUNTER_BYTES:].fill_(0xFF)
    for c in (many, few, many):
        check_window(c, run_window(pkv, c, 2400, 4, ws), 2400, 4, str(len(c.lens)))


@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 4), ("f16", 64, 8), ("f32", 128, 2)])
def test_split_by_batch_and_bound(pkv, dtype, D, G):
    """The same sequence by itself, in a batch and under larger bounds, each of which splits it in its own
    way: every one within the bound of the exact values, and the same bits on a second call."""
    for lens, bounds in (((5000,), (5000, 40000, 1 << 20)), ((5000, 40, 0, 4999, 128, 700, 1, 2500), (5000, 40000))):
        c = Cache(lens, 2, G, D, 16, dtype, seed=7)
        c.bt = np.concatenate([c.bt, np.full((len(lens), 1 << 16), -1, np.int32)], 1)
        c.tables = torch.from_numpy(c.bt).to(DEV)
        for n in bounds:
            out = run_window(pkv, c, 4500, 4, max_len=n)
            check_window(c, out, 4500, 4, f"bound {n}")
            assert torch.equal(out, run_window(pkv, c, 4500, 4, max_len=n))
            got = [torch.full((len(lens), 2, n), float("nan"), device=DEV) for _ in range(2)]
            outs = [run_scores(pkv, c, None, x, max_len=n) for x in got]
            check_scores(c, outs[0], None, got[0], f"bound {n}")
            assert torch.equal(*outs) and torch.equal(*(torch.nan_to_num(x, -1.0) for x in got))
