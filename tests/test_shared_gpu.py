"""Decode of groups that share a prefix against the float64 definition, element by
element within the bound that the roundings allow."""
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


def problem(sizes, pre, lens, H_q, H_kv, D, BS, seed):
    """Caches whose rows past the ends hold NaN; (tensors, numpy views)."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = [list(pre), list(lens)]
    pages = [[-(-n // BS) for n in r] for r in rows]
    total = sum(map(sum, pages))
    ids = rng.permutation(total + 2)
    k, v = (torch.randn(total + 2, H_kv, BS, D, generator=g, device="cuda").to(torch.bfloat16)
            for _ in range(2))
    at, tables = 0, []
    for r, pg in zip(rows, pages):
        t = np.full((len(r), max(1, max(pg, default=1)) + 1), ids[-1], dtype=np.int64)
        for i, (n, m) in enumerate(zip(r, pg)):
            t[i, :m] = ids[at:at + m]
            at += m
            if n % BS:
                for c in (k, v):
                    c[int(t[i, m - 1]), :, n % BS:] = float("nan")
        tables.append(t)
    for c in (k, v):
        c[ids[-2:].copy()] = float("nan")
    q = torch.randn(len(lens), H_q, D, generator=g, device="cuda").to(torch.bfloat16)
    gi = np.concatenate([[0], np.cumsum(sizes)])
    return (q, k, v, i32(gi), i32(tables[0]), i32(pre), i32(tables[1]), i32(lens)), \
        (gi, tables[0], pre, tables[1], lens)


def check(sizes, pre, lens, H_q, H_kv, D, BS, seed, softcap=0.0, alibi=False, scale=None):
    t, (gi, pt, pre, bt, lens) = problem(sizes, pre, lens, H_q, H_kv, D, BS, seed)
    scale = float(np.float32(1 / np.sqrt(D) if scale is None else scale))
    slopes = np.array([2.0 ** (-8.0 * (h + 1) / H_q) for h in range(H_q)], dtype=np.float32)
    out = pa.paged_attn_decode_shared(*t, scale, softcap=softcap,
                                      alibi_slopes=torch.tensor(slopes).cuda() if alibi else None)
    torch.cuda.synchronize()
    res = serving.attend_shared(*(serving.bf16_to_f64(x) for x in t[:3]), gi, pt, pre, bt, lens,
                                scale, softcap, slopes.astype(np.float64) if alibi else None)
    # sequences past the last group have no prefix
    free = int(gi[-1])
    if free < len(lens):
        solo = serving.attend(*(serving.bf16_to_f64(x) for x in t[:3]), None, bt, lens, scale,
                              softcap=softcap, slopes=slopes.astype(np.float64) if alibi else None)
        res.out[free:], res.tol[free:] = solo.out[free:], solo.tol[free:]
    got = serving.bf16_to_f64(out)
    assert np.isfinite(got).all()
    err = np.abs(got - res.out)
    over = np.divide(err, res.tol, out=np.where(err > 0, np.inf, 0.0), where=res.tol > 0)
    assert over.max() <= 1.0, (over.max(), np.unravel_index(over.argmax(), over.shape))
    return out, t, scale


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("BS", [16, 32])
@pytest.mark.parametrize("H_q,H_kv", [(2, 2), (8, 2), (12, 2), (16, 1)])
def test_groups_of_every_size(D, BS, H_q, H_kv):
    check([1, 5, 0, 9, 2], [40, 257, 16, 1000, 1], [3, 0, 1, 16, 17, 40, 100, 5, 1, 0, 33, 31, 2, 70,
                                                    8, 9, 300], H_q, H_kv, D, BS, D + H_q)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kw", [dict(softcap=30.0), dict(alibi=True), dict(softcap=2.0, alibi=True)])
def test_score_options(D, kw):
    check([7, 3], [500, 77], [1, 2, 30, 100, 0, 16, 17, 5, 1, 64], 8, 2, D, 16, D + 1, **kw)


def test_a_group_wider_than_a_row_tile():
    check([150, 3], [700, 33], list(np.random.default_rng(3).integers(0, 60, size=153)), 8, 2, 128,
          16, 5)
    check([90], [300], list(np.random.default_rng(4).integers(0, 60, size=90)), 6, 1, 256, 16, 6)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=30.0), dict(softcap=2.0, alibi=True)])
def test_as_many_pieces_as_the_gpu_has_places(D, kw):
    """The two-team kernel: full pieces, and a group of one short piece."""
    check([290, 8], [333, 140], list(np.random.default_rng(5).integers(0, 40, size=300)), 128, 8,
          D, 16, 12 + D, **kw)


def test_empty_prefixes_empty_tails_and_sequences_in_no_group():
    out, _, _ = check([2, 2, 3], [0, 50, 0], [0, 4, 0, 3, 1, 0, 2, 90, 0], 4, 2, 64, 16, 7)
    assert torch.count_nonzero(out[0]) == 0 and torch.count_nonzero(out[8]) == 0
    check([], [], [5, 20], 4, 2, 128, 16, 8)


def test_long_prefix_is_split():
    check([4], [20011], [5, 600, 0, 33], 6, 1, 256, 16, 9)
    check([3], [30001], [5, 600, 1], 8, 1, 128, 32, 10, alibi=True)
    check([2], [9000], [0, 0], 4, 1, 64, 16, 11)


def test_equals_the_decode_of_joined_tables():
    """Whole-block prefixes: the plain decode of tables that begin with the prefix's blocks."""
    pre, lens, BS = [64, 160], [5, 30, 17, 1, 48], 16
    t, (gi, pt, _, bt, _) = problem([2, 3], pre, lens, 8, 2, 128, BS, 12)
    maxb = 16
    joined = np.zeros((5, maxb), dtype=np.int64)
    total = []
    for s in range(5):
        g = 0 if s < 2 else 1
        a, b = pre[g] // BS, -(-lens[s] // BS)
        joined[s, :a], joined[s, a:a + b] = pt[g, :a], bt[s, :b]
        total.append(pre[g] + lens[s])
    a = pa.paged_attn_decode_shared(*t, 0.09)
    b = pa.paged_attn_decode(t[0], t[1], t[2], i32(joined), i32(total), 0.09)
    # each within (2 eps + eps) of the values' mean magnitude (below 1 here) plus 1e-4
    assert (a.float() - b.float()).abs().max() <= 6 * 2.0 ** -8 + 2e-4


def test_repeat_calls_and_a_captured_one_are_bitwise_identical():
    out, t, scale = check([9, 4], [3000, 100], [30] * 13, 8, 2, 128, 16, 13)
    assert torch.equal(out, pa.paged_attn_decode_shared(*t, scale))
    n = pa.paged_attn_shared_workspace_bytes(13, 2, 8, 2, 128, t[6].shape[1], 16)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    dst = torch.zeros_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(pa.PagedAttnError, match="workspace"):
            pa.paged_attn_decode_shared(*t, scale, out=dst)
        pa.paged_attn_decode_shared(*t, scale, out=dst, workspace=ws)
    for _ in range(2):
        dst.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dst, out)


def test_bad_prefix_blocks_are_reported():
    t, (gi, pt, pre, bt, lens) = problem([2], [100], [5, 6], 4, 2, 128, 16, 14)
    status = i32([0])
    nb = t[1].shape[0]
    try:
        pa.paged_attn_set_checks(nb, status)
        pa.paged_attn_decode_shared(*t, 0.1)
        torch.cuda.synchronize()
        assert int(status) == 0
        bad = t[4].clone()
        bad[0, 2] = nb + 7
        pa.paged_attn_decode_shared(*t[:4], bad, *t[5:], 0.1)
        torch.cuda.synchronize()
        assert int(status) == 1
    finally:
        pa.paged_attn_set_checks(0, None)


def test_one_workspace_serves_every_entry_point_in_any_order():
    t, (gi, pt, pre, bt, lens) = problem([3, 2], [3000, 100], [30, 2000, 5, 1, 700], 8, 2, 128, 16,
                                         15)
    q, k, v, _, _, _, own, n = t
    qo = i32([0, 1, 2, 3, 4, 5])
    calls = [
        lambda ws: pa.paged_attn_decode_shared(*t, 0.1, workspace=ws),
        lambda ws: pa.paged_attn_decode_mods(q, k, v, own, n, 0.1, workspace=ws),
        lambda ws: pa.paged_attn_decode_multi_mods(q, k, v, qo, own, n, 0.1, workspace=ws),
    ]
    need = max(pa.paged_attn_shared_workspace_bytes(5, 2, 8, 2, 128, own.shape[1], 16),
               pa.paged_attn_mods_workspace_bytes(5, 8, 2, 128, own.shape[1], 16),
               pa.paged_attn_multi_mods_workspace_bytes(5, 5, 8, 2, 128, own.shape[1], 16))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    expect = [c(torch.zeros_like(ws)) for c in calls]
    for order in ((0, 1, 2), (2, 1, 0), (2, 0, 1), (1, 2, 0)):
        for i in order:
            for w in (ws, None):
                assert torch.equal(calls[i](w), expect[i])
