"""Attention of drafted trees against the float64 definition, element by element within the
bound that the roundings allow, with NaN in every cache row that no row of its sequence
sees."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_decode_gb300 as pa
import workloads
from oracle import serving, speculative

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


def slopes_of(H):
    return np.array([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=np.float32)


def tree_bits(rng, m, kind):
    """[m, m]: `tree` (random parents), `chain`, `any` (no tree at all), `padded` (a tree whose last
    third and every fifth node is padding), `none`."""
    bits = np.zeros((m, m), dtype=bool)
    if kind == "any":
        return rng.random((m, m)) < 0.3
    if kind == "none":
        return bits
    pad = np.zeros(m, dtype=bool)
    if kind == "padded":
        pad = (np.arange(m) % 5 == 4) | (np.arange(m) >= m - m // 3)
    for j in range(m):
        if pad[j]:
            continue
        p = j - 1 if kind == "chain" else int(rng.integers(-1, j)) if j else -1
        if p >= 0 and not pad[p]:
            bits[j] = bits[p]
        bits[j, j] = True
    return bits


def within(out, res, what=""):
    got = serving.bf16_to_f64(out)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    err = np.abs(got - res.out)
    over = np.divide(err, res.tol, out=np.where(err > 0, np.inf, 0.0), where=res.tol > 0)
    at = np.unravel_index(over.argmax(), over.shape)
    assert over.max() <= 1.0, f"{what}: {over.max():.3f} of the bound at {at}"


def make(lens, qlens, H_q, H_kv, D, BS, seed, kind="tree", window=0, prefix=None, words=None, gain=1.0):
    """lens count the drafted tokens (fewer than qlens: some drafted ones are before the first)."""
    spec = workloads.custom_spec("tree", len(lens), H_q, H_kv, D, BS, [max(n, 1) for n in lens])
    w = workloads.make(spec, seed=seed, device="cuda", poison="nan")
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    qo = np.concatenate([[0], np.cumsum(qlens)])
    q = (torch.randn(int(qo[-1]), H_q, D, generator=g) * gain).to(torch.bfloat16).cuda()
    words = words or max(1, -(-max(qlens) // 32))
    kinds = [kind] if isinstance(kind, str) else kind
    mask = np.zeros((int(qo[-1]), words), dtype=np.int32)
    bt = w.block_tables.cpu().numpy()
    for s, (n, m) in enumerate(zip(lens, qlens)):
        bits = tree_bits(rng, m, kinds[s % len(kinds)])
        mask[qo[s]:qo[s + 1]] = speculative.mask_words(bits, words)
        ctx = n - m
        bits[:, 32 * words:] = False
        pos = ctx + (bits & (ctx + np.arange(m) >= 0)).sum(1) - 1
        seen = np.zeros(max(n, 0), dtype=bool)
        for t in range(max(ctx, 0)):
            first = prefix is not None and t < prefix[s % len(prefix)]
            seen[t] = (m > 0) and (first or not window or bool((t > pos - window).any()))
        for j in range(m):
            if ctx + j >= 0:
                seen[ctx + j] = bits[:, j].any()
        for t in np.nonzero(~seen)[0]:
            for c in (w.k_cache, w.v_cache):
                c[int(bt[s, t // BS]), :, t % BS] = float("nan")
    w.seq_lens.copy_(i32(lens))
    return w, q, qo, mask, bt


def run_case(lens, qlens, H_q, H_kv, D, BS, seed, softcap=0.0, alibi=False, window=0, prefix=None,
             scale=None, workspace=None, **kw):
    w, q, qo, mask, bt = make(lens, qlens, H_q, H_kv, D, BS, seed, window=window, prefix=prefix, **kw)
    scale = w.scale if scale is None else scale
    prefix = None if prefix is None else np.resize(np.asarray(prefix), len(lens))
    slopes = slopes_of(H_q)
    out = torch.full_like(q, 7.0)
    pa.paged_attn_decode_tree(
        q, w.k_cache, w.v_cache, i32(qo), i32(mask), w.block_tables, w.seq_lens, scale,
        softcap=softcap, alibi_slopes=torch.tensor(slopes).cuda() if alibi else None, window=window,
        prefix_lens=None if prefix is None else i32(prefix), out=out, workspace=workspace)
    torch.cuda.synchronize()
    res = speculative.attend_tree(
        serving.bf16_to_f64(q), serving.bf16_to_f64(w.k_cache), serving.bf16_to_f64(w.v_cache), qo, mask,
        bt, lens, float(np.float32(scale)), softcap=softcap,
        slopes=slopes.astype(np.float64) if alibi else None, window=window, prefix_lens=prefix)
    within(out, res, f"D{D} BS{BS} G{H_q // H_kv}")
    return out


@pytest.mark.parametrize("D,BS", [(64, 16), (128, 16), (128, 32), (256, 16), (256, 32)])
@pytest.mark.parametrize("ctx,m,G", [(0, 1, 1), (0, 7, 4), (1, 1, 8), (57, 7, 4), (63, 2, 4),
                                     (100, 31, 4), (64, 32, 4), (200, 33, 2), (127, 64, 4), (40, 65, 5),
                                     (300, 100, 1)])
def test_row_and_token_tiles(D, BS, ctx, m, G):
    run_case([ctx + m], [m], 2 * G, 2, D, BS, ctx + m)


LENS = [1, 15, 40, 17, 33, 100, 257, 0, 700, 64, 129, 50]
QLENS = [1, 3, 16, 0, 33, 70, 13, 0, 64, 64, 100, 7]
KINDS = ["tree", "padded", "any", "chain", "tree", "padded", "none"]


@pytest.mark.parametrize("D,BS,H_q,H_kv", [(64, 16, 4, 2), (128, 16, 4, 1), (128, 32, 6, 2), (256, 16, 6, 1),
                                           (64, 32, 16, 1)])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=30.0), dict(softcap=0.5), dict(alibi=True),
                                dict(window=1), dict(window=16), dict(window=150), dict(prefix=[3, 140, 0]),
                                dict(softcap=50.0, alibi=True, window=45, prefix=[0, 5, 33, 200])])
def test_ragged_batches_with_every_option(D, BS, H_q, H_kv, kw):
    run_case(LENS, QLENS, H_q, H_kv, D, BS, 5, kind=KINDS, **kw)


@pytest.mark.parametrize("D,H_q,H_kv", [(64, 8, 2), (128, 8, 2), (256, 4, 1)])
@pytest.mark.parametrize("kw", [dict(), dict(alibi=True), dict(window=20, softcap=5.0)])
def test_trees_of_up_to_256_tokens(D, H_q, H_kv, kw):
    run_case([700, 256, 300, 255], [256, 256, 200, 255], H_q, H_kv, D, 16, 9, kind=["tree", "chain", "padded"], **kw)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_more_drafted_tokens_than_bits_or_than_tokens(D):
    """Tokens past the words are seen by no row; tokens before the sequence's first are none."""
    run_case([100, 300], [70, 290], 4, 2, D, 16, 3, kind="any", words=2)
    run_case([5, 20, 0], [9, 60, 4], 4, 2, D, 16, 4, kind=["chain", "tree"])
    run_case([5, 20], [9, 60], 4, 2, D, 16, 4, kind=["chain", "any"], alibi=True, window=7)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_two_teams_and_split_ranges(D):
    """Enough rows for pieces of 256, and few enough sequences for parts."""
    run_case([300 + 7 * s for s in range(90)], [64 - s % 30 for s in range(90)], 8, 2, D, 16, 11, kind=KINDS)
    run_case([5000], [40], 8, 2, D, 16, 12, kind="padded")
    run_case([5000], [5], 4, 1, D, 32, 13, softcap=20.0, window=3000, prefix=[100])


@pytest.mark.parametrize("D,H_q,H_kv", [(64, 16, 4), (128, 32, 8), (128, 8, 8), (256, 12, 4)])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0, window=900), dict(alibi=True, prefix=[300, 5])])
def test_long_sequences_among_many_short_ones(D, H_q, H_kv, kw):
    """Pieces for every SM, a few of them much longer; the same bits every time."""
    lens = [100 + s for s in range(70)]
    lens[3], lens[40], lens[41], lens[69] = 3000, 2111, 900, 1500
    outs = [run_case(lens, [40 - s % 23 for s in range(70)], H_q, H_kv, D, 16, 21, kind=KINDS, **kw) for _ in range(3)]
    assert all(torch.equal(outs[0], o) for o in outs)


@pytest.mark.parametrize("D,H_q,H_kv", [(64, 8, 1), (128, 4, 2), (256, 6, 1)])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=9.0, window=12, prefix=[3])])
def test_more_sequences_than_are_ranked(D, H_q, H_kv, kw):
    n = 150
    run_case([(7 * s) % 61 for s in range(n)], [min((7 * s) % 61, (5 * s) % 23) for s in range(n)], H_q, H_kv, D, 16, 22,
             kind=KINDS, **kw)


def test_two_graphs_that_share_a_workspace():
    """Captured apart, replayed in any order, with the parts of one larger than the other's."""
    calls = []
    for lens, ql, seed in (([900], [20], 31), ([400, 70], [40, 3], 32)):
        w, q, qo, mask, bt = make(lens, ql, 8, 2, 128, 16, seed)
        calls.append((q, w.k_cache, w.v_cache, i32(qo), i32(mask), w.block_tables, w.seq_lens, w.scale))
    need = max(pa.paged_attn_tree_workspace_bytes(len(c[6]), c[0].shape[0], 8, 2, 128, c[5].shape[1], 16) for c in calls)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    want = [pa.paged_attn_decode_tree(*c) for c in calls]
    outs = [torch.empty_like(x) for x in want]
    torch.cuda.synchronize()
    graphs = []
    for c, out in zip(calls, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.paged_attn_decode_tree(*c, out=out, workspace=ws)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (1, 1), (0, 0)):
        for out in outs:
            out.zero_()
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize()
        for k in set(order):
            assert torch.equal(outs[k], want[k])


@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_other_scales(scale):
    run_case([200], [30], 4, 2, 128, 16, 14, scale=scale)


def test_a_chain_equals_the_causal_call():
    lens, ql = [300 + s for s in range(200)], [32 - s % 9 for s in range(200)]  # (the same pieces, not split)
    w, q, qo, mask, bt = make(lens, ql, 8, 2, 128, 16, 15, kind="chain")
    a = pa.paged_attn_decode_tree(q, w.k_cache, w.v_cache, i32(qo), i32(mask), w.block_tables, w.seq_lens, w.scale)
    b = pa.paged_attn_decode_multi_mods(q, w.k_cache, w.v_cache, i32(qo), w.block_tables, w.seq_lens, w.scale)
    assert torch.equal(a, b)


def test_rows_outside_the_offsets_are_left():
    w, q, qo, mask, bt = make([50, 60], [5, 9], 8, 2, 128, 16, 16)
    more = torch.cat([q[:3], q, q[:4]])
    m2 = np.concatenate([mask[:3], mask, mask[:4]])
    out = torch.full_like(more, 3.0)
    pa.paged_attn_decode_tree(more, w.k_cache, w.v_cache, i32(qo + 3), i32(m2), w.block_tables, w.seq_lens, w.scale,
                              out=out)
    ref = pa.paged_attn_decode_tree(q, w.k_cache, w.v_cache, i32(qo), i32(mask), w.block_tables, w.seq_lens, w.scale)
    assert torch.equal(out[3:17], ref) and (out[:3] == 3).all() and (out[17:] == 3).all()


def test_captured_replayed_on_another_stream_with_new_trees():
    w, q, qo, mask, bt = make([200, 90], [20, 31], 8, 2, 128, 16, 17)
    need = pa.paged_attn_tree_workspace_bytes(2, q.shape[0], 8, 2, 128, w.block_tables.shape[1], 16)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    d_mask, d_qo, out = i32(mask), i32(qo), torch.empty_like(q)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        with pytest.raises(pa.PagedAttnError):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                pa.paged_attn_decode_tree(q, w.k_cache, w.v_cache, d_qo, d_mask, w.block_tables, w.seq_lens, w.scale, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            pa.paged_attn_decode_tree(q, w.k_cache, w.v_cache, d_qo, d_mask, w.block_tables, w.seq_lens, w.scale, out=out,
                                      workspace=ws)
    for kind in ("tree", "any"):
        rng = np.random.default_rng(18)
        new = np.concatenate([speculative.mask_words(tree_bits(rng, m, kind), mask.shape[1]) for m in (20, 31)])
        for c in (w.k_cache, w.v_cache):
            c[torch.isnan(c)] = 0.0
        d_mask.copy_(i32(new))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        res = speculative.attend_tree(serving.bf16_to_f64(q), serving.bf16_to_f64(w.k_cache), serving.bf16_to_f64(w.v_cache),
                                      qo, new, bt, [200, 90], float(np.float32(w.scale)))
        within(out, res, kind)


def test_checks_report_bad_blocks_and_too_many_drafted_tokens():
    w, q, qo, mask, bt = make([50, 60], [5, 40], 8, 2, 128, 16, 19, words=1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = w.block_tables.clone()
    bad[0, 1] = w.k_cache.shape[0]
    try:
        pa.paged_attn_set_checks(w.k_cache.shape[0], status)
        pa.paged_attn_decode_tree(q, w.k_cache, w.v_cache, i32(qo), i32(mask), bad, w.seq_lens, w.scale)
    finally:
        pa.paged_attn_set_checks(0, None)
    assert int(status) == 3
