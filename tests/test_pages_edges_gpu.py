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


# ------------------------------------------------------------------ several batches of a CTA

@pytest.mark.parametrize("n", [256, 257, 512, 513, 600, 1000])
@pytest.mark.parametrize("H,BS,D,fp8", [(2, 16, 128, False), (5, 32, 128, True)])
def test_lists_of_several_batches(n, H, BS, D, fp8):
    """A CTA looks up 256 entries of an accepted list at a time; rows that move by one place take those of the
    next batch before it begins."""
    m = n + 5
    lists = [np.arange(1, n + 1), np.arange(n), np.arange(5, m), np.r_[np.arange(250), np.arange(255, m)][:n],
             np.sort(np.random.default_rng(n).permutation(m)[:n])]
    lens = [m + 3 + 7 * s for s in range(len(lists))]
    pages = [-(-x // BS) for x in lens]
    nb, maxb = sum(pages) + 1, max(pages)
    ids = np.random.default_rng(1).permutation(nb)
    bt, at = np.full((len(lists), maxb), -1), 0
    for s, x in enumerate(pages):
        bt[s, :x] = ids[at:at + x]
        at += x
    g = torch.Generator(device="cuda").manual_seed(n)
    if fp8:
        k, v = (torch.randint(0, 256, (nb, H, BS, D), generator=g, device="cuda", dtype=torch.uint8) for _ in "kv")
        kw = dict(k_scale=torch.randn(nb, H, BS, generator=g, device="cuda"),
                  v_scale=torch.randn(nb, H, BS, generator=g, device="cuda"))
    else:
        k, v = (torch.randn(nb, H, BS, D, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
        kw = {}
    want = [t.clone() for t in (k, v, *kw.values())]
    for t in want:
        for s, x in enumerate(lists):
            ctx = lens[s] - m
            old, new = (ctx + torch.tensor(y) for y in (x, np.arange(n)))
            row = torch.tensor(bt[s])
            rows = t[row[old // BS], :, old % BS].clone()
            t[row[new // BS], :, new % BS] = rows
    out = pa.paged_kv_compact(k, v, i32(np.arange(len(lists) + 1) * m), i32(np.array(lists)), i32(bt), i32(lens), **kw)
    assert out.cpu().tolist() == [x - m + n for x in lens]
    assert all(torch.equal(a, b) for a, b in zip((k, v, *kw.values()), want))


@pytest.mark.parametrize("forks,H", [(511, 1), (512, 1), (513, 1), (100001, 1), (100001, 2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_forks_of_several_batches(forks, H, in_place):
    """A CTA looks up 512 forks at a time; past 512 forks for each SM it has several batches of them."""
    BS, D, parents = 16, 64, 40
    rng = np.random.default_rng(forks)
    lens = rng.integers(0, 3 * BS + 1, size=parents)
    par, kid = rng.integers(0, parents, size=forks), parents + rng.permutation(forks)
    need = lens[par] % BS > 0
    nb = 3 * parents + int(need.sum()) + 3
    bt = np.full((parents + forks, 3), -1)
    bt[:parents] = np.arange(3 * parents).reshape(parents, 3)
    stack = 3 * parents + rng.permutation(nb - 3 * parents)
    g = torch.Generator(device="cuda").manual_seed(forks)
    k, v = (torch.randn(nb, H, BS, D, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
    full, tail = lens // BS, lens % BS
    fresh = np.full(forks, -1)
    fresh[need] = stack[len(stack) - 1 - np.arange(need.sum())]
    refs, want_bt, want_lens = np.zeros(nb, dtype=np.int64), bt.copy(), np.r_[lens, np.zeros(forks, dtype=np.int64)]
    want_lens[kid] = lens[par]
    for j in range(3):
        some = full[par] > j
        want_bt[kid[some], j] = bt[par[some], j]
        np.add.at(refs, bt[par[some], j], 1)
    want_bt[kid[need], full[par[need]]] = fresh[need]
    want = []
    for t in (k, v):
        w, rows = t.clone(), torch.arange(BS, device="cuda")
        src, dst = (torch.tensor(x[need], device="cuda") for x in (bt[par, np.minimum(full[par], 2)], fresh))
        keep = (rows[None] < torch.tensor(tail[par[need]], device="cuda")[:, None])[:, None, :, None]
        w[dst] = torch.where(keep, w[src], w[dst])
        want.append(w)
    d_bt, d_lens, d_refs = i32(bt), i32(np.r_[lens, np.zeros(forks, dtype=np.int64)]), i32(np.zeros(nb))
    count, refused = i32([len(stack)]), i32([-1])
    left = pa.paged_kv_fork(k, v, d_bt, d_lens, i32(par), i32(kid), d_refs, i32(stack), count, refused=refused,
                            free_count_out=count if in_place else None)
    assert int(left) == len(stack) - need.sum() and int(refused) == 0
    for got, x in ((d_bt, want_bt), (d_lens, want_lens), (d_refs, refs)):
        assert np.array_equal(got.cpu().numpy(), x)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
