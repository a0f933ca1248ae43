"""Block assignment and the append by slot against their definitions: exact, over
page sizes, request lengths around page borders, refusals and many sequences."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_decode_gb300 as pa
from oracle import serving

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


def problem(seed, lens, new, BS, spare=7, maxb=None):
    rng = np.random.default_rng(seed)
    lens, new = np.asarray(lens), np.asarray(new)
    held = -(-np.maximum(lens, 0) // BS)
    total = -(-np.maximum(lens + np.maximum(new, 0), 0) // BS)
    maxb = int(total.max()) + 2 if maxb is None else maxb
    need = int((total - held).clip(min=0).sum())
    table = np.full((len(lens), maxb), -7, dtype=np.int64)
    ids = rng.permutation(int(held.sum()) + need + spare)
    at = 0
    for s, h in enumerate(held):
        h = min(int(h), maxb)
        table[s, :h] = ids[at:at + h]
        at += h
    return lens, new, table, ids[at:]


def check(lens, new, table, free, count, BS, max_new, in_place=False):
    expect = serving.assign(lens, new, table, free, count, BS, max_new)
    d_lens, d_table, d_count = i32(lens), i32(table), i32([count])
    refused = i32([-1])
    guard = torch.full((max_new + 16,), 77, dtype=torch.int64, device="cuda")
    kw = dict(seq_lens_out=d_lens, free_count_out=d_count) if in_place else {}
    lens_out, qo, slots, left = pa.paged_kv_assign(
        d_lens, i32(new), d_table, i32(free), d_count, BS, max_new, refused=refused,
        slot_map=guard[:max_new], **kw)
    torch.cuda.synchronize()
    got = (lens_out, qo, slots, left, refused, d_table)
    names = ("seq_lens", "qo_indptr", "slot_map", "free_count", "refused", "block_tables")
    for name, g, e in zip(names, got, expect):
        np.testing.assert_array_equal(g.cpu().numpy().reshape(-1), np.asarray(e).reshape(-1), name)
    assert (guard[max_new:] == 77).all()
    if not in_place:  # the inputs are left alone
        np.testing.assert_array_equal(d_lens.cpu().numpy(), lens)
        assert int(d_count) == count


@pytest.mark.parametrize("BS", [16, 32])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n", [1, 3, 33, 1000, 1025, 5000])
def test_decode_step(BS, in_place, n):
    rng = np.random.default_rng(n + BS)
    lens = rng.integers(0, 5 * BS, size=n)
    lens[0] = BS            # a full page: the new token opens one
    lens[-1] = BS - 1
    p = problem(n, lens, np.ones(n, dtype=int), BS)
    check(*p, len(p[3]), BS, n, in_place)


@pytest.mark.parametrize("BS", [16, 32])
@pytest.mark.parametrize("in_place", [False, True])
def test_prompts_of_every_size(BS, in_place):
    rng = np.random.default_rng(5)
    new = np.concatenate([np.arange(0, 70), rng.integers(0, 4000, size=90), [0, 0, 1]])
    lens = np.concatenate([np.zeros(35, dtype=int), rng.integers(0, 100, size=len(new) - 35)])
    p = problem(6, lens, new, BS)
    check(*p, len(p[3]), BS, int(new.sum()) + 37, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("max_new", [0, 1, 50, 20000])
def test_no_sequences(in_place, max_new):
    none = np.zeros(0, dtype=int)
    check(none, none, np.zeros((0, 4), dtype=int), np.arange(9), 9, 16, max_new, in_place)


@pytest.mark.parametrize("short", [0, 1, 5, 40, 10 ** 6])
def test_too_few_free_blocks(short):
    rng = np.random.default_rng(short)
    lens, new = rng.integers(0, 200, size=60), rng.integers(0, 90, size=60)
    lens, new, table, free = problem(7, lens, new, 16, spare=0)
    check(lens, new, table, free, max(0, len(free) - short), 16, int(new.sum()))


def test_refusals_of_single_sequences():
    lens = np.array([5, 30, -3, 64, 10, 0, 47])
    new = np.array([3, 40, 2, 1, -1, 0, 1])    # 1: past its row; 2, 4: negative; 3: row is full
    lens, new, table, free = problem(8, lens, new, 16, maxb=4)
    check(lens, new, table, free, len(free), 16, 64)
    check(lens, new, table, free, len(free), 16, 20)   # the rows of 1 and what follows do not fit
    check(lens, new, table, free, len(free), 16, 0)


def test_counts_outside_the_stack_are_clamped():
    lens, new, table, free = problem(9, [3, 17], [20, 20], 16)
    check(lens, new, table, free, len(free) + 50, 16, 40)
    check(lens, new, table, free, -4, 16, 40)


def test_a_chain_of_captured_steps():
    """Five replays of one captured in-place step: the lengths grow, the stack shrinks."""
    n, BS, maxb = 9, 16, 6
    lens, table = np.arange(9) * 5, np.full((n, maxb), -1, dtype=np.int64)
    held = -(-lens // BS)
    for s in range(n):
        table[s, :held[s]] = 100 + np.arange(held[s]) + 10 * s
    free, new = np.arange(40)[::-1].copy(), np.array([1, 0, 16, 3, 1, 1, 2, 1, 7])
    d_lens, d_table, d_count = i32(lens), i32(table), i32([40])
    d_new, d_free = i32(new), i32(free)
    qo, slots = i32(np.zeros(n + 1)), torch.zeros(40, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.paged_kv_assign(d_lens, d_new, d_table, d_free, d_count, BS, 40, seq_lens_out=d_lens,
                           qo_indptr=qo, slot_map=slots, free_count_out=d_count)
    count = 40
    for _ in range(5):
        lens, eqo, eslots, count, _, table = serving.assign(lens, new, table, free, count, BS, 40)
        graph.replay()
        torch.cuda.synchronize()
        for g, e in ((d_lens, lens), (qo, eqo), (slots, eslots), (d_table, table)):
            np.testing.assert_array_equal(g.cpu().numpy(), e)
        assert int(d_count) == count


def test_bad_ids_are_reported():
    lens, new, table, free = problem(10, [3, 17], [20, 20], 16)
    status = i32([0])
    try:
        pa.paged_attn_set_checks(int(free.max()), status)  # the largest id is outside
        free = np.concatenate([np.sort(free)])
        pa.paged_kv_assign(i32(lens), i32(new), i32(table), i32(free), i32([len(free)]), 16, 40)
        torch.cuda.synchronize()
    finally:
        pa.paged_attn_set_checks(0, None)
    assert int(status) == 1


# ---------------------------------------------------------------- append by slot

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("BS", [16, 32])
@pytest.mark.parametrize("H_kv,rows,fused", [(1, 1, False), (2, 7, True), (3, 100, True),
                                             (8, 1500, True), (8, 513, False)])
def test_append_slots(D, BS, H_kv, rows, fused):
    g = torch.Generator(device="cuda").manual_seed(D + rows)
    nb = -(-rows // BS) + 5
    rng = np.random.default_rng(rows)
    slots = rng.permutation(nb * BS)[:rows]
    slots[rng.random(rows) < 0.1] = -1
    if rows > 50:
        slots[3], slots[4], slots[5] = nb * BS, 2 ** 40, -2 ** 40   # outside: skipped
    wide = torch.randn(rows, 5 * H_kv * D, generator=g, device="cuda").to(torch.bfloat16)
    cut = [wide[:, i * H_kv * D:(i + 1) * H_kv * D].unflatten(1, (H_kv, D)) for i in (2, 4)]
    k_new, v_new = cut if fused else [c.contiguous() for c in cut]
    caches = [torch.randn(nb, H_kv, BS, D, generator=g, device="cuda").to(torch.bfloat16)
              for _ in range(2)]
    expect = [c.clone() for c in caches]
    for r, s in enumerate(slots):
        if 0 <= s < nb * BS:
            expect[0][s // BS, :, s % BS] = k_new[r]
            expect[1][s // BS, :, s % BS] = v_new[r]
    pa.paged_kv_append_slots(k_new, v_new, *caches,
                             torch.tensor(slots, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    for got, e in zip(caches, expect):
        assert torch.equal(got.view(torch.int16), e.view(torch.int16))


def test_append_slots_past_the_pool_are_reported():
    k = torch.ones(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(3, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    status = i32([0])
    try:
        pa.paged_attn_set_checks(3, status)
        for slots, bit in (([-1, 4], 0), ([48, 4], 1)):
            pa.paged_kv_append_slots(k, k, cache, cache.clone(),
                                     torch.tensor(slots, dtype=torch.int64, device="cuda"))
            assert int(status) == bit
    finally:
        pa.paged_attn_set_checks(0, None)


def test_assigned_slots_equal_the_append_along_the_tables():
    """assign -> append by slot writes the bytes that the append through lengths and
    tables writes."""
    BS, H_kv, D = 16, 2, 128
    lens, new, table, free = problem(11, [0, 15, 16, 33, 7], [20, 1, 1, 30, 0], BS)
    d_lens, d_table = i32(lens), i32(table)
    nb = int(max(table.max(), free.max())) + 1
    rows = int(new.sum())
    lens2, qo, slots, _ = pa.paged_kv_assign(d_lens, i32(new), d_table, i32(free),
                                             i32([len(free)]), BS, rows)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(rows, H_kv, D, generator=g, device="cuda").to(torch.bfloat16)
            for _ in range(2))
    a = [torch.zeros(nb, H_kv, BS, D, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    pa.paged_kv_append_slots(k, v, a[0], a[1], slots)
    pa.paged_kv_append_multi(k, v, a[2], a[3], qo, d_table.clamp(min=0), lens2)
    torch.cuda.synchronize()
    assert torch.equal(a[0], a[2]) and torch.equal(a[1], a[3])
    assert torch.count_nonzero(a[0]) > 0
