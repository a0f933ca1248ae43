"""The float64 definitions of trees, rotation and page handling, pinned by what they must
equal: other definitions, closed forms and conserved quantities."""
import numpy as np
import pytest

from oracle import serving, speculative as sp

SCALE = 0.2


def problem(rng, lens, H_q, H_kv, D=8, BS=4, spare=3):
    pages = [-(-n // BS) for n in lens]
    total = sum(pages) + spare
    ids = rng.permutation(total)
    bt = np.zeros((len(lens), max(pages) + 1), dtype=np.int64)
    at = 0
    for s, n in enumerate(pages):
        bt[s, :n] = ids[at:at + n]
        at += n
    k, v = rng.standard_normal((2, total, H_kv, BS, D))
    return k, v, bt


@pytest.mark.parametrize("kw", [dict(), dict(softcap=1.5), dict(window=5), dict(prefix_lens=[2, 0, 1]),
                                dict(slopes=np.array([0.5, 0.25, 0.1, 0.02]))])
def test_a_chain_is_the_causal_attention_of_several_tokens(kw):
    rng = np.random.default_rng(1)
    lens, ql = [9, 14, 3], [3, 6, 3]
    k, v, bt = problem(rng, lens, 4, 2)
    qo = np.concatenate([[0], np.cumsum(ql)])
    q = rng.standard_normal((qo[-1], 4, 8))
    bits = np.concatenate([np.tril(np.ones((m, 6), dtype=bool))[:m] for m in ql])
    bits[:, :] &= np.arange(6) <= np.concatenate([np.arange(m) for m in ql])[:, None]
    window = kw.get("window", 0)
    if window:  # a window bounds the cached tokens alone: here it also holds the whole chain
        assert window >= 5
        kw = dict(kw, window=8)
    a = sp.attend_tree(q, k, v, qo, sp.mask_words(bits, 1), bt, lens, SCALE, **kw)
    b = serving.attend(q, k, v, qo, bt, lens, SCALE, **kw)
    assert np.abs(a.out - b.out).max() < 1e-12


def test_each_path_of_a_tree_is_a_sequence_of_its_own():
    rng = np.random.default_rng(2)
    ctx, parent = 5, [-1, 0, 0, 1, 2, -1]
    m = len(parent)
    k, v, bt = problem(rng, [ctx + m], 2, 1)
    q = rng.standard_normal((m, 2, 8))
    bits = np.zeros((m, m), dtype=bool)
    for j, p in enumerate(parent):
        if p >= 0:
            bits[j] = bits[p]
        bits[j, j] = True
    slopes = np.array([0.3, 0.1])
    out = sp.attend_tree(q, k, v, [0, m], sp.mask_words(bits, 2), bt, [ctx + m], SCALE, slopes=slopes).out
    K, V = (serving.rows_of(x, bt[0], ctx + m) for x in (k, v))
    for j in range(m):
        keep = np.concatenate([np.arange(ctx), ctx + np.nonzero(bits[j])[0]])
        kp, vp = K[None, keep].transpose(0, 2, 1, 3), V[None, keep].transpose(0, 2, 1, 3)
        ref = serving.attend(q[j:j + 1], kp, vp, None, np.zeros((1, 1), dtype=int), [len(keep)], SCALE,
                             slopes=slopes).out
        assert np.abs(out[j] - ref[0]).max() < 1e-12


def test_mask_words_round_trip_and_bits_past_the_words():
    rng = np.random.default_rng(3)
    bits = rng.random((5, 70)) < 0.5
    assert (sp.mask_bits(sp.mask_words(bits, 3), 70) == bits).all()
    assert not sp.mask_bits(sp.mask_words(bits, 2), 70)[:, 64:].any()


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance_alone(inter):
    rng = np.random.default_rng(4)
    D, R = 16, 16
    angle = np.arange(50)[:, None] * 100.0 ** (-np.arange(R // 2) / (R // 2))
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    a, b = rng.standard_normal((2, 1, 1, D))
    dots = []
    for p, r in ((3, 10), (20, 27)):
        x, _ = sp.turn(a, None, 0.0, [np.array([p])], [0] * 8, cs, inter)
        y, _ = sp.turn(b, None, 0.0, [np.array([r])], [0] * 8, cs, inter)
        assert np.isclose((x * x).sum(), (a * a).sum())
        dots.append((x * y).sum())
    assert np.isclose(dots[0], dots[1])


def test_norm_axes_and_the_part_that_does_not_turn():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 2, 16))
    cs = np.zeros((4, 8))
    cs[:, :4] = np.cos(np.arange(4))[:, None]
    cs[:, 4:] = np.sin(np.arange(4))[:, None]
    w = rng.standard_normal(16)
    pos = np.array([[0, 1, 2], [3, 0, 9]])  # 9 is clamped to 3
    z, _ = sp.turn(x, w, 1e-6, pos, [0, 1, 5, 0], cs, False)  # axis 5 is clamped to 1
    y = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-6) * w
    assert np.allclose(z[..., 8:], y[..., 8:])
    for i, axis in enumerate([0, 1, 1, 0]):
        p = np.minimum(pos[axis], 3)[:, None]
        assert np.allclose(z[..., i], y[..., i] * np.cos(p) - y[..., i + 4] * np.sin(p))
        assert np.allclose(z[..., i + 4], y[..., i + 4] * np.cos(p) + y[..., i] * np.sin(p))


def test_compaction_on_the_contiguous_tokens():
    rng = np.random.default_rng(6)
    lens, ql = [10, 7, 6, 4], [6, 3, 6, 0]
    k, _, bt = problem(rng, lens, 1, 2)
    acc = np.array([[1, 2, 5, -1], [0, 1, 2, -1], [2, 1, 4, 5], [0, -1, -1, -1]])
    out, new = sp.compact(k, np.concatenate([[0], np.cumsum(ql)]), acc, bt, lens)
    kept = [[1, 2, 5], [0, 1, 2], [2], []]  # the third list falls, the fourth tree is empty
    assert list(new) == [4 + 3, 4 + 3, 1, 4]
    for s, n in enumerate(lens):
        old, got = serving.rows_of(k, bt[s], n), serving.rows_of(out, bt[s], n)
        ctx = n - ql[s]
        assert (got[:ctx] == old[:ctx]).all()
        for i, j in enumerate(kept[s]):
            assert (got[ctx + i] == old[ctx + j]).all()


def test_forks_and_releases_conserve_the_blocks():
    rng = np.random.default_rng(7)
    BS, nb, rows, maxb = 4, 60, 8, 6
    free = list(rng.permutation(nb))
    bt, lens = np.full((rows, maxb), -1, dtype=np.int64), np.zeros(rows, dtype=np.int64)
    k = rng.standard_normal((nb, 1, BS, 2))
    for s, n in enumerate((9, 8, 3)):
        for j in range(-(-n // BS)):
            bt[s, j] = free.pop()
        lens[s] = n
    refs, stack, count = np.zeros(nb, dtype=np.int64), np.full(nb, -1), len(free)
    stack[:count] = free
    (k2,), bt, lens, refs, count, refused = sp.fork([k], bt, lens, [0, 0, 1, 2, 9], [3, 4, 5, 6, 7], refs,
                                                    stack, count)
    assert refused == 1 and list(lens) == [9, 8, 3, 9, 9, 8, 3, 0]
    for p, c in ((0, 3), (0, 4), (1, 5), (2, 6)):
        assert (serving.rows_of(k2, bt[c], lens[c]) == serving.rows_of(k, bt[p], lens[p])).all()
        if lens[p] % BS:
            assert bt[c, lens[p] // BS] != bt[p, lens[p] // BS]
    held = [[bt[s, j] for j in range(-(-lens[s] // BS))] for s in range(rows)]
    for b in range(nb):  # counted once less than held; free exactly where not held
        n = sum(h.count(b) for h in held)
        assert refs[b] == max(n - 1, 0) and (b in stack[:count]) == (n == 0)
    keep = [5, 8, 0, 0, 9, 0, 3, 0]
    lens, refs, stack, count = sp.release(bt, lens, keep, refs, stack, count, BS)
    held = [[bt[s, j] for j in range(-(-lens[s] // BS))] for s in range(rows)]
    for b in range(nb):
        n = sum(h.count(b) for h in held)
        assert refs[b] == max(n - 1, 0) and list(stack[:count]).count(b) == (n == 0)


def test_release_order_and_a_full_stack():
    bt = np.array([[5, 6, 7], [5, 8, 9]])
    lens, refs, stack, count = sp.release(bt, [12, 10], [0, 4], [0] * 5 + [1] + [0] * 9, [1, -1, -1, -1, -1],
                                          1, 4)
    assert list(lens) == [0, 4] and refs[5] == 0
    assert list(stack) == [1, 6, 7, 8, 9] and count == 5
    _, _, stack, count = sp.release(bt, [12, 10], [0, 4], None, [1, -1, -1], 1, 4)
    assert list(stack) == [1, 5, 6] and count == 3
