"""Compaction, forks and release at the edges of their ranges: index ranges, several batches of a CTA, calls
against their contract."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_decode_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_decode_gb300 import build

    build.build()
    pa.load()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bad", [False, True])
def test_release_of_a_table_that_just_fits_its_keys(bad):
    """2^31 - 2 entries, all released: places and batches next to the end of 32 bits.  With an entry that is no
    block the ranks are counted instead of known."""
    n, maxb = 42966, 49981
    bt = torch.arange(n * maxb, dtype=torch.int32, device="cuda").view(n, maxb)
    if bad:
        bt[7, 3] = -1
    lens = torch.full((n,), maxb * 16, dtype=torch.int32, device="cuda")
    stack = torch.full((n * maxb,), -2, dtype=torch.int32, device="cuda")
    out, left = pa.paged_kv_release(bt, lens, torch.zeros_like(lens), stack, i32([0]), 16)
    torch.cuda.synchronize()
    assert int(left) == n * maxb - bad and not out.any()
    at = 7 * maxb + 3 if bad else n * maxb
    flat = bt.view(-1)
    assert torch.equal(stack[:at], flat[:at])
    if bad:
        assert torch.equal(stack[at:-1], flat[at + 1:]) and int(stack[-1]) == -2


@pytest.mark.parametrize("parents,children,want", [
    ([0, 0, 1], [2, 3, 4], 0), ([0, 2], [2, 3], 2), ([2, 0], [3, 2], 2), ([0, 1], [3, 3], 2),
    ([0] * 600 + [599], list(range(1, 601)) + [601], 2), ([0] * 600, list(range(1, 601)), 0),
    ([0] * 600, list(range(1, 600)) + [1], 2), ([0, 7], [3, -1], 2),
])
def test_children_that_are_parents_or_twice_children_are_reported(parents, children, want):
    """All rows hold the same token counts and pages of the pool, whichever is read first."""
    rows = 602
    k, v = (torch.zeros(640, 1, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bt, lens = i32([[0, 1]] * rows), i32([20] * rows)
    refs, free, status = i32([0] * 640), i32(range(2, 640)), i32([0])
    try:
        pa.paged_attn_set_checks(640, status)
        pa.paged_kv_fork(k, v, bt, lens, i32(parents), i32(children), refs, free, i32([638]))
        torch.cuda.synchronize()
    finally:
        pa.paged_attn_set_checks(0, None)
    assert int(status) == want
