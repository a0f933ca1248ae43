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
