"""Compaction, forks and release against their definitions: whole numbers and copied rows, so
everything is equal bit for bit."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_decode_gb300 as pa
from oracle import speculative as sp

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


class Cache:
    """Random bits (bf16 NaN among them), so that a copied row is told from any other."""

    def __init__(self, nb, H, BS, D, fp8, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        if fp8:
            make = lambda: torch.randint(0, 256, (nb, H, BS, D), generator=g, device="cuda", dtype=torch.uint8)
            self.kw = dict(k_scale=torch.randn(nb, H, BS, generator=g, device="cuda"),
                           v_scale=torch.randn(nb, H, BS, generator=g, device="cuda"))
        else:
            make = lambda: torch.randint(-2 ** 15, 2 ** 15, (nb, H, BS, D), generator=g, device="cuda",
                                         dtype=torch.int16).view(torch.bfloat16)
            self.kw = {}
        self.k, self.v = make(), make()

    def host(self):
        bits = lambda t: t.cpu().view(torch.int16).numpy() if t.dtype is torch.bfloat16 else t.cpu().numpy()
        return [bits(t).copy() for t in (self.k, self.v, *self.kw.values())]


def tables(rng, lens, BS, maxb, spare=3):
    pages = [-(-n // BS) for n in lens]
    nb = sum(pages) + spare
    ids = rng.permutation(nb)
    bt = np.full((len(lens), maxb), -7, dtype=np.int64)
    at = 0
    for s, n in enumerate(pages):
        bt[s, :n] = ids[at:at + n]
        at += n
    return bt, nb, ids[at:]


SHAPES = [(1, 16, 64, False), (2, 16, 128, False), (8, 32, 128, False), (3, 16, 256, False), (2, 16, 128, True),
          (5, 32, 256, True)]


# ------------------------------------------------------------------ compaction

def check_compact(lens, qlens, accepted, shape, seed=0, maxb=None):
    H, BS, D, fp8 = shape
    rng = np.random.default_rng(seed)
    maxb = maxb or max(1, -(-max(lens) // BS)) + 1
    bt, nb, _ = tables(rng, lens, BS, maxb)
    c = Cache(nb, H, BS, D, fp8, seed)
    qo = np.concatenate([[0], np.cumsum(qlens)])
    want = [sp.compact(x, qo, accepted, bt, lens) for x in c.host()]
    out = pa.paged_kv_compact(c.k, c.v, i32(qo), i32(accepted), i32(bt), i32(lens), **c.kw)
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), want[0][1])
    for got, (x, _) in zip(c.host(), want):
        assert np.array_equal(got, x)


def random_lists(rng, qlens, most, depth):
    acc = np.full((len(qlens), most), -1, dtype=np.int64)
    for s, m in enumerate(qlens):
        n = int(rng.integers(0, min(m, depth, most) + 1))
        acc[s, :n] = np.sort(rng.permutation(m)[:n])
    return acc


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("most,depth", [(1, 1), (8, 8), (70, 70)])
def test_compaction(shape, most, depth):
    rng = np.random.default_rng(most)
    lens = [1, 64, 70, 100, 300, 257, 0, 90]
    qlens = [1, 64, 3, 33, 64, 70, 0, 16]
    check_compact(lens, qlens, random_lists(rng, qlens, most, depth), shape, seed=most)


@pytest.mark.parametrize("shape", SHAPES)
def test_rows_that_take_each_others_places(shape):
    """Every row moves one or a few places: each place written is read by another row first."""
    m = 200
    lists = [np.arange(1, m), np.arange(0, m, 2), np.arange(m), np.arange(37, m), [m - 1], [0], []]
    acc = np.full((len(lists), m), -1, dtype=np.int64)
    for s, x in enumerate(lists):
        acc[s, :len(x)] = x
    check_compact([m + 13 + s for s in range(len(lists))], [m] * len(lists), acc, shape)


def test_lists_that_end_early():
    acc = [[3, 2, 4, 5], [0, 0, 1, 2], [1, 4, 2, 3], [-1, 0, 1, 2], [2, 7, 8, 9], [-5, 1, 2, 3], [6, -1, 7, 8]]
    check_compact([50] * 7, [10, 10, 10, 10, 7, 10, 10], np.array(acc), SHAPES[1])


def test_more_drafted_tokens_than_tokens_and_no_list():
    check_compact([5, 20, 3], [9, 20, 50], np.array([[0, 5, 8], [1, 2, 19], [46, 47, 49]]), SHAPES[1])
    check_compact([5, 20], [2, 20], np.zeros((2, 0), dtype=int), SHAPES[1])


def test_bad_blocks_move_nothing_and_are_reported():
    H, BS, D, _ = SHAPES[1]
    c = Cache(6, H, BS, D, False, 1)
    before = c.host()
    status = i32([0])
    try:
        pa.paged_attn_set_checks(6, status)
        out = pa.paged_kv_compact(c.k, c.v, i32([0, 8]), i32([[3, 4, -1]]), i32([[6, 0, 1]]), i32([12]))
    finally:
        pa.paged_attn_set_checks(0, None)
    assert int(out) == 6 and int(status) == 1
    assert all(np.array_equal(a, b) for a, b in zip(c.host(), before))


# ------------------------------------------------------------------ forks

def check_fork(lens, rows, parents, children, shape, seed=0, free_count=None, in_place=False, spare=None, refs=None,
               extra=2):
    H, BS, D, fp8 = shape
    rng = np.random.default_rng(seed)
    held = np.zeros(rows, dtype=np.int64)
    held[:len(lens)] = lens
    maxb = max(1, -(-max(lens) // BS)) + extra
    bt, nb, free = tables(rng, held, BS, maxb, spare=len(parents) + 5 if spare is None else spare)
    c = Cache(nb, H, BS, D, fp8, seed)
    count = len(free) if free_count is None else free_count
    refs = rng.integers(0, 4, size=nb)
    want = sp.fork(c.host(), bt, held, parents, children, refs, free, count)
    d_bt, d_lens, d_refs, d_count, refused = i32(bt), i32(held), i32(refs), i32([count]), i32([-1])
    left = pa.paged_kv_fork(c.k, c.v, d_bt, d_lens, i32(parents), i32(children), d_refs, i32(free), d_count,
                            free_count_out=d_count if in_place else None, refused=refused, **c.kw)
    torch.cuda.synchronize()
    assert int(refused) == want[5] and int(left) == want[4]
    for got, x in ((d_bt, want[1]), (d_lens, want[2]), (d_refs, want[3])):
        assert np.array_equal(got.cpu().numpy(), x)
    for got, x in zip(c.host(), want[0]):
        assert np.array_equal(got, x)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_forks(shape, in_place):
    lens = [1, 16, 17, 100, 64, 300, 31]
    check_fork(lens, 20, [0, 0, 1, 2, 3, 3, 3, 4, 5, 6, 6], [7, 19, 8, 10, 9, 11, 12, 13, 15, 14, 18], shape,
               in_place=in_place)


@pytest.mark.parametrize("count", [0, 1, 3, -4])
def test_forks_without_enough_blocks(count):
    check_fork([5, 16, 40, 33], 9, [0, 1, 2, 3, 0], [4, 5, 6, 7, 8], SHAPES[1], free_count=count)


def test_forks_of_rows_that_are_none_and_of_empty_rows():
    check_fork([20, 0, 40], 8, [0, 8, -1, 2, 1, 2, 2], [4, 5, 6, 2, 7, 9, -3], SHAPES[1])
    check_fork([20], 3, [], [], SHAPES[1])


@pytest.mark.parametrize("n", [255, 256, 257, 700])
def test_many_forks(n):
    rng = np.random.default_rng(n)
    parents = 9
    check_fork([int(x) for x in rng.integers(0, 90, size=parents)] , parents + n, rng.integers(0, parents, size=n),
               parents + rng.permutation(n), SHAPES[0], free_count=n // 2)
    check_fork([int(x) for x in rng.integers(0, 90, size=parents)], parents + n, rng.integers(0, parents, size=n),
               parents + rng.permutation(n), SHAPES[0], in_place=True)


def test_forks_with_bad_blocks_are_reported():
    c = Cache(6, 2, 16, 128, False, 1)
    before = c.host()
    bt, lens, refs, status = i32([[9, 1], [0, 0], [0, 0]]), i32([20, 0, 0]), i32([0] * 6), i32([0])
    try:
        pa.paged_attn_set_checks(6, status)
        left = pa.paged_kv_fork(c.k, c.v, bt, lens, i32([0]), i32([2]), refs, i32([3, 77]), i32([2]))
    finally:
        pa.paged_attn_set_checks(0, None)
    assert int(status) == 1 and int(left) == 1
    assert bt.cpu().tolist() == [[9, 1], [0, 0], [9, 77]] and lens.cpu().tolist() == [20, 0, 20]
    assert refs.cpu().tolist() == [0] * 6 and all(np.array_equal(a, b) for a, b in zip(c.host(), before))


# ------------------------------------------------------------------ release

def check_release(bt, lens, keep, refs, stack, count, BS, in_place=False):
    want = sp.release(np.asarray(bt), lens, keep, refs, stack, count, BS)
    d_lens, d_count, d_stack = i32(lens), i32([count]), i32(stack)
    d_refs = None if refs is None else i32(refs)
    out, left = pa.paged_kv_release(i32(bt), d_lens, i32(keep), d_stack, d_count, BS, block_refs=d_refs,
                                    seq_lens_out=d_lens if in_place else None,
                                    free_count_out=d_count if in_place else None)
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), want[0]) and int(left) == want[3]
    assert np.array_equal(d_stack.cpu().numpy(), want[2])
    if refs is not None:
        assert np.array_equal(d_refs.cpu().numpy(), want[1])


def random_release(n, most, BS, share, seed, cut):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, most + 1, size=n)
    maxb = -(-most // BS) + 1
    bt, nb, _ = tables(rng, lens, BS, maxb)
    pages = -(-lens // BS)
    for s in range(n):  # groups hold their first one's pages together
        a = s // share * share
        m = min(pages[s], pages[a])
        bt[s, :m] = bt[a, :m]
    used = np.concatenate([bt[s, :pages[s]] for s in range(n)]) if n else np.zeros(0, dtype=np.int64)
    refs = np.maximum(np.bincount(used.astype(np.int64), minlength=nb) - 1, 0)
    keep = np.where(rng.random(n) < 0.4, 0, lens - rng.integers(0, cut + 1, size=n))
    keep[rng.random(n) < 0.1] = most + 99
    return bt, lens, keep, refs, nb


@pytest.mark.parametrize("BS", [16, 32])
@pytest.mark.parametrize("n,most,share", [(1, 40, 1), (3, 100, 1), (40, 300, 3), (257, 1000, 4), (1500, 200, 7),
                                          (9, 20000, 2), (3000, 64, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_release_of_shared_blocks(BS, n, most, share, in_place):
    bt, lens, keep, refs, nb = random_release(n, most, BS, share, n + BS, 50)
    stack = np.full(nb + 4, -1)
    check_release(bt, lens, keep, refs, stack, 2, BS, in_place)


@pytest.mark.parametrize("share", [1, 3, None])
@pytest.mark.parametrize("in_place", [False, True])
def test_release_of_very_many_blocks(share, in_place):
    """More entries than the threads hold at once."""
    bt, lens, keep, refs, nb = random_release(700, 13000, 16, share or 1, 4, 0)
    keep = np.where(np.arange(700) % 50 == 7, lens // 2, 0)
    assert (-(-lens // 16) - -(-np.minimum(keep, lens) // 16)).sum() > 16 * 1024 * 8
    check_release(bt, lens, keep, refs if share else None, np.full(nb, -1), 0, 16, in_place)


@pytest.mark.parametrize("n,most", [(1, 40), (100, 500), (2000, 100)])
def test_release_without_counts(n, most):
    bt, lens, keep, _, nb = random_release(n, most, 16, 1, n, 30)
    bt[::3, 1] = -1  # passed over
    check_release(bt, lens, keep, None, np.full(nb, -1), 0, 16)


def test_release_of_nothing_and_of_no_sequences():
    check_release([[1, 2], [3, 4]], [20, 17], [20, 17], [0] * 5, [-1] * 4, 1, 16)
    check_release(np.zeros((0, 4), dtype=int), [], [], [0] * 5, [-1] * 4, 1, 16, True)


def test_one_block_in_many_entries():
    """More entries than holders counted, the same block twice in one row, counts that stay."""
    bt = [[4, 4, 5], [4, 5, 6], [6, 4, 9]]
    check_release(bt, [48] * 3, [0, 0, 0], [0, 0, 0, 0, 3, 1, 5, 0, 0, 0], [-1] * 10, 0, 16)
    check_release(bt, [48] * 3, [16, 0, 33], [0, 0, 0, 0, 9, 1, 0, 0, 0, 0], [-1] * 10, 0, 16)
    check_release([[2] * 3] * 700, [48] * 700, [0] * 700, [0, 0, 2099], [-1] * 4, 0, 16)
    check_release([[2] * 3] * 700, [48] * 700, [0] * 700, [0, 0, 2100], [-1] * 4, 0, 16)


def test_a_full_stack_and_bad_entries_are_reported():
    status = i32([0])
    stack, count = i32([-1, -1, -1]), i32([2])
    try:
        pa.paged_attn_set_checks(8, status)
        _, left = pa.paged_kv_release(i32([[3, 4, 5]]), i32([48]), i32([0]), stack, count, 16, block_refs=i32([0] * 8))
        assert int(status) == 2 and int(left) == 3 and stack.cpu().tolist() == [-1, -1, 3]
        status.zero_()
        stack, refs = i32([-1] * 4), i32([0] * 8)
        _, left = pa.paged_kv_release(i32([[3, 8, -1]]), i32([48]), i32([0]), stack, i32([0]), 16, block_refs=refs)
        assert int(status) == 1 and int(left) == 1 and stack.cpu().tolist() == [3, -1, -1, -1]
        status.zero_()
        out, _ = pa.paged_kv_release(i32([[3, 4, 5]]), i32([49]), i32([-3]), i32([-1] * 4), i32([0]), 16)
        assert int(status) == 2 and int(out) == 0
    finally:
        pa.paged_attn_set_checks(0, None)


@pytest.mark.parametrize("n", [600])
def test_the_order_of_the_stack_is_always_the_same(n):
    bt, lens, keep, refs, nb = random_release(n, 800, 16, 5, 3, 10)
    seen = None
    for _ in range(10):
        stack, d_refs = torch.full((nb,), -1, dtype=torch.int32, device="cuda"), i32(refs)
        pa.paged_kv_release(i32(bt), i32(lens), i32(keep), stack, i32([0]), 16, block_refs=d_refs)
        assert seen is None or torch.equal(stack, seen)
        seen = stack
