"""Calls at the edges of what the serving entry points allow, on the GPU."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_decode_gb300 as pa
import workloads
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


def test_no_groups_in_a_captured_stream():
    """A batch without shared prefixes: a workspace of the size that is asked for serves the
    captured call, whose output is the decode's."""
    w = workloads.make(workloads.custom_spec("none", 3, 8, 2, 128, 16, [5, 700, 33]), device="cuda")
    n = pa.paged_attn_shared_workspace_bytes(3, 0, 8, 2, 128, w.max_blocks_per_seq, 16)
    assert n >= pa.paged_attn_workspace_bytes(3, 8, 2, 128, w.max_blocks_per_seq, 16) > 0
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    none = (i32([0]), torch.zeros(0, 4, dtype=torch.int32, device="cuda"),
            torch.zeros(0, dtype=torch.int32, device="cuda"))
    out = torch.zeros_like(w.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.paged_attn_decode_shared(w.q, w.k_cache, w.v_cache, *none, w.block_tables, w.seq_lens,
                                    w.scale, out=out, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, pa.paged_attn_decode_mods(w.q, w.k_cache, w.v_cache, w.block_tables,
                                                      w.seq_lens, w.scale))


def f64(t):
    return serving.bf16_to_f64(t)


def within(out, res):
    got = f64(out)
    assert np.isfinite(got).all()
    err = np.abs(got - res.out)
    over = np.divide(err, res.tol, out=np.where(err > 0, np.inf, 0.0), where=res.tol > 0)
    assert over.max() <= 1.0, (over.max(), np.unravel_index(over.argmax(), over.shape))


# ---- documents that begin behind a query (a blanked or padding row of a packed chunk)
def check_documents(lens, qlens, H_q, H_kv, D, BS, docs, seed, causal=True, softcap=0.0,
                    alibi=False, window=0, prefix=None):
    """docs: one start per query row, anywhere.  K and V rows that no query of the sequence
    sees are NaN."""
    w = workloads.make(workloads.custom_spec("docs", len(lens), H_q, H_kv, D, BS, lens), seed=seed,
                       device="cuda", poison="nan")
    qo = np.concatenate([[0], np.cumsum(qlens)])
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(int(qo[-1]), H_q, D, generator=g).to(torch.bfloat16).cuda()
    docs = np.asarray(docs, dtype=np.int64)
    bt = w.block_tables.cpu().numpy()
    hidden = 0
    for s, (n, m) in enumerate(zip(lens, qlens)):
        seen = serving.visible(n - m + np.arange(m), n, causal, window,
                               0 if prefix is None else prefix[s], docs[qo[s]:qo[s + 1]])
        for t in np.nonzero(~seen.any(axis=0))[0]:
            for c in (w.k_cache, w.v_cache):
                c[int(bt[s, t // BS]), :, t % BS] = float("nan")
            hidden += 1
    slopes = np.array([2.0 ** (-8.0 * (h + 1) / H_q) for h in range(H_q)], dtype=np.float32)
    out = pa.paged_attn_decode_multi_mods(
        q, w.k_cache, w.v_cache, i32(qo), w.block_tables, w.seq_lens, w.scale, causal=causal,
        softcap=softcap, alibi_slopes=torch.tensor(slopes).cuda() if alibi else None,
        window=window, prefix_lens=None if prefix is None else i32(prefix), doc_starts=i32(docs))
    torch.cuda.synchronize()
    within(out, serving.attend(f64(q), f64(w.k_cache), f64(w.v_cache), qo, bt, lens,
                               float(np.float32(w.scale)), causal=causal, softcap=softcap,
                               slopes=slopes.astype(np.float64) if alibi else None, window=window,
                               prefix_lens=prefix, doc_starts=docs))
    return hidden


def test_tokens_between_the_documents_that_nobody_sees():
    # rows 1 to 9 of a chunk see nothing, and nobody sees their tokens
    assert check_documents([21], [11], 4, 2, 128, 16, [0] + [21] * 9 + [20], 1) == 9
    # one blanked row in the middle of a prompt, the next document behind it
    docs = [0] * 50 + [100] + [51] * 49
    assert check_documents([100], [100], 4, 2, 128, 16, docs, 2) == 1
    assert check_documents([100], [100], 4, 2, 128, 16, docs, 3, prefix=[51]) == 0
    # a row that sees nothing before rows whose own document begins earlier: seen by those
    assert check_documents([100], [100], 4, 2, 128, 16, [0] * 50 + [100] + [7] * 49, 4) == 0


@pytest.mark.parametrize("D,BS,H_q,H_kv", [(64, 16, 4, 2), (128, 32, 6, 2), (256, 16, 2, 2),
                                           (64, 32, 32, 8), (128, 16, 32, 8)])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0), dict(alibi=True), dict(window=7),
                                dict(prefix=[3, 0, 40, 33]), dict(causal=False)])
def test_documents_that_begin_anywhere(D, BS, H_q, H_kv, kw):
    lens, qlens = [300, 33, 170, 700], [300, 20, 129, 257]
    rng = np.random.default_rng(D + BS + H_q)
    docs = []
    for n, m in zip(lens, qlens):
        pos = n - m + np.arange(m)
        start = np.maximum(0, pos - rng.integers(0, 40, size=m))
        blank = rng.random(m) < 0.4
        docs.append(np.where(blank, rng.integers(pos + 1, n + 5), start))
    hidden = check_documents(lens, qlens, H_q, H_kv, D, BS, np.concatenate(docs), 5, **kw)
    assert hidden > 20 or kw.get("causal") is False


def test_hidden_tokens_of_a_range_in_parts():
    docs = np.zeros(40, dtype=int)
    docs[5:30] = 2 ** 31 - 1
    docs[30:] = 8991
    check_documents([9001], [40], 2, 1, 128, 16, docs, 6)
    check_documents([9001], [40], 2, 1, 256, 32, docs, 7, window=5000)


@pytest.mark.parametrize("H_q,H_kv", [(2, 1), (32, 16)])
def test_hidden_tokens_of_many_sequences(H_q, H_kv):
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 120, size=300)
    qlens = np.minimum(rng.integers(0, 60, size=300), lens)
    docs = np.concatenate([np.where(rng.random(m) < 0.5, n, np.maximum(0, n - m + np.arange(m) - 2))
                           for n, m in zip(lens, qlens)])
    assert check_documents(list(lens), list(qlens), H_q, H_kv, 64, 16, docs, 8) > 100


# ---- a NaN in a query or in a token that it sees reaches the output, however the work is cut
def nan_rows(out):
    """[rows, heads]: all NaN or all finite, true for NaN."""
    bad = torch.isnan(out)
    assert torch.equal(bad.all(-1), bad.any(-1))
    return bad.all(-1).cpu().numpy()


LONG = [7, 20000, 1, 40]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[7, 30, 1, 40], LONG])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=30.0), dict(window=15000)])
def test_a_nan_query_of_a_decode(D, lens, kw):
    w = workloads.make(workloads.custom_spec("nanq", 4, 8, 2, D, 16, lens), device="cuda")
    w.q[1, 2] = float("nan")
    w.q[2] = float("nan")
    expect = np.zeros((4, 8), dtype=bool)
    expect[1, 2] = expect[2] = True
    args = (w.k_cache, w.v_cache, w.block_tables, w.seq_lens, w.scale)
    assert np.array_equal(nan_rows(pa.paged_attn_decode_mods(w.q, *args, **kw)), expect)
    if not kw:
        assert np.array_equal(nan_rows(pa.paged_attn_decode(w.q, *args)), expect)
    if D > 64:
        f = workloads.to_fp8(w)
        a8 = (w.q, f.k8, f.v8, f.k_scale, f.v_scale, w.block_tables, w.seq_lens, w.scale)
        assert np.array_equal(nan_rows(pa.paged_attn_decode_fp8_mods(*a8, **kw)), expect)
        if not kw:
            assert np.array_equal(nan_rows(pa.paged_attn_decode_fp8(*a8)), expect)


@pytest.mark.parametrize("D,H_q,H_kv", [(64, 8, 2), (128, 8, 2), (256, 8, 2), (64, 64, 32),
                                        (128, 64, 32)])
@pytest.mark.parametrize("lens", [[7, 300, 1, 40], LONG])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=30.0), dict(window=15000), dict(alibi=True)])
def test_a_nan_query_among_many(D, H_q, H_kv, lens, kw):
    w = workloads.make(workloads.custom_spec("nanm", 4, H_q, H_kv, D, 16, lens), device="cuda")
    qo = np.cumsum([0, 3, 9, 1, 40])
    q = torch.randn(53, H_q, D, device="cuda").to(torch.bfloat16)
    q[5, 2] = float("nan")
    q[12] = float("nan")
    expect = np.zeros((53, H_q), dtype=bool)
    expect[5, 2] = expect[12] = True
    kw = dict(kw)
    if kw.pop("alibi", False):
        kw["alibi_slopes"] = torch.full((H_q,), 2.0 ** -6, device="cuda")
    args = (q, w.k_cache, w.v_cache, i32(qo), w.block_tables, w.seq_lens, w.scale)
    assert np.array_equal(nan_rows(pa.paged_attn_decode_multi_mods(*args, **kw)), expect)
    if not kw and H_q == 8:
        assert np.array_equal(nan_rows(pa.paged_attn_decode_multi(*args, 40)), expect)
    # a blanked query sees nothing: a zero row whatever it holds
    docs = np.zeros(53, dtype=int)
    docs[12] = 2 ** 31 - 1
    out = pa.paged_attn_decode_multi_mods(*args, **kw, doc_starts=i32(docs))
    expect[12] = False
    assert np.array_equal(nan_rows(out), expect) and torch.count_nonzero(out[12]) == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("own", [[0, 5, 700, 40], [3, 9000, 1, 0]])
def test_a_nan_query_over_a_shared_prefix(D, own):
    w = workloads.make(workloads.custom_spec("nans", 5, 8, 2, D, 16, own + [5000]), device="cuda")
    w.q[1, 2] = float("nan")
    w.q[3] = float("nan")
    expect = np.zeros((4, 8), dtype=bool)
    expect[1, 2] = expect[3] = True
    for members in (4, 2):  # the others have no prefix
        out = pa.paged_attn_decode_shared(w.q[:4].contiguous(), w.k_cache, w.v_cache,
                                          i32([0, members]), w.block_tables[4:].clone(),
                                          i32([5000]), w.block_tables[:4].clone(), i32(own),
                                          w.scale)
        if members == 2:
            expect[3] = own[3] > 0  # without a token a zero row
        assert np.array_equal(nan_rows(out), expect)


def test_a_nan_token_reaches_those_who_see_it():
    w = workloads.make(workloads.custom_spec("nank", 2, 8, 2, 128, 16, [20000, 50]), device="cuda")
    w.k_cache[int(w.block_tables[0, 19000 // 16]), 1, 19000 % 16] = float("nan")
    expect = np.zeros((2, 8), dtype=bool)
    expect[0, 4:] = True
    args = (w.k_cache, w.v_cache, w.block_tables, w.seq_lens, w.scale)
    assert np.array_equal(nan_rows(pa.paged_attn_decode(w.q, *args)), expect)
    assert np.array_equal(nan_rows(pa.paged_attn_decode_mods(w.q, *args)), expect)
    assert not nan_rows(pa.paged_attn_decode_mods(w.q, *args, window=999)).any()
    q = torch.randn(8, 8, 128, device="cuda").to(torch.bfloat16)
    out = pa.paged_attn_decode_multi_mods(q, w.k_cache, w.v_cache, i32([0, 6, 8]), *args[2:],
                                          softcap=5.0)
    assert np.array_equal(nan_rows(out), np.repeat(expect, [6, 2], axis=0))


# ---- the early prologue begins when all but the launch just ahead is complete
@pytest.mark.parametrize("between", ["decode", "mods", "early"])
def test_early_prologue_two_launches_behind_an_append(between):
    """An append, a decode of other caches, then with the early prologue a decode that
    reads the appended rows: it may find the launch just ahead running, not the append."""
    sp = workloads.custom_spec("chain", 64, 8, 8, 128, 16, [256] * 64)
    w = workloads.make(sp, device="cuda")
    other = workloads.make(workloads.custom_spec("other", 1, 8, 8, 128, 16, [20]), device="cuda")
    bt = w.block_tables.long()
    t = torch.arange(256, device="cuda")
    slots = (bt[:, t // 16] * 16 + t % 16).reshape(-1).contiguous()

    def decode(x, fn=pa.paged_attn_decode):
        return fn(x.q, x.k_cache, x.v_cache, x.block_tables, x.seq_lens, x.scale)

    decode(w), decode(other, pa.paged_attn_decode_mods)
    for i in range(20):
        rows = torch.randn(2, slots.numel(), 8, 128, device="cuda").to(torch.bfloat16)
        torch.cuda.synchronize()
        try:
            if between == "early":
                pa.paged_attn_set_launch_flags(pa.FLAG_EARLY_PROLOGUE)
            pa.paged_kv_append_slots(rows[0], rows[1], w.k_cache, w.v_cache, slots)
            decode(other, pa.paged_attn_decode_mods if between == "mods" else pa.paged_attn_decode)
            pa.paged_attn_set_launch_flags(pa.FLAG_EARLY_PROLOGUE)
            out = decode(w)
        finally:
            pa.paged_attn_set_launch_flags(0)
        torch.cuda.synchronize()
        assert torch.equal(out, decode(w)), i


# ---- the library's own workspaces
def test_streams_side_by_side_without_workspaces():
    """Split work of every entry point on several streams at once, and grown buffers."""
    ws = [workloads.make(workloads.custom_spec("side", 3, 8, 2, 128, 16, lens), seed=i,
                         device="cuda") for i, lens in enumerate(([9000, 5, 300], [20, 8000, 7000],
                                                                  [4000, 4000, 4000]))]
    qo = i32([0, 4, 5, 9])

    def calls(w):
        g = torch.Generator(device="cuda").manual_seed(w.seed)
        q = torch.randn(9, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
        args = (w.k_cache, w.v_cache)
        rest = (w.block_tables, w.seq_lens, w.scale)
        lone = (i32([0, 3]), w.block_tables[:1].clone(), w.seq_lens[:1].clone())
        return [lambda: pa.paged_attn_decode_mods(w.q, *args, *rest, softcap=30.0),
                lambda: pa.paged_attn_decode_multi_mods(q, *args, qo, *rest),
                lambda: pa.paged_attn_decode_shared(w.q, *args, *lone, *rest)]

    work = [calls(w) for w in ws]
    torch.cuda.synchronize()
    expect = [[c() for c in cs] for cs in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = [[] for _ in work]
    for i in range(12):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append((work[k][(i + k) % 3](), (i + k) % 3))
    torch.cuda.synchronize()
    for k, outs in enumerate(got):
        for out, which in outs:
            assert torch.equal(out, expect[k][which])


# ---- block ids outside the pool, with checks on: reported, and read as pages of zeros
def with_checks(num_blocks, call):
    status = i32([0])
    pa.paged_attn_set_checks(num_blocks, status)
    try:
        out = call()
        torch.cuda.synchronize()
    finally:
        pa.paged_attn_set_checks(0, None)
    return out, int(status)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_bad_page_is_a_page_of_zeros(D):
    lens, qlens = [100, 40], [20, 3]
    w = workloads.make(workloads.custom_spec("bad", 2, 8, 2, D, 16, lens), device="cuda")
    qo = np.cumsum([0] + qlens)
    q = torch.randn(23, 8, D, device="cuda").to(torch.bfloat16)
    bt = w.block_tables.cpu().numpy()
    scale = float(np.float32(w.scale))
    bad = w.block_tables.clone()
    bad[0, 5] = w.num_blocks + 3
    skipped = w.block_tables.clone()
    skipped[0, 0] = -9                      # ahead of the window
    k0, v0 = w.k_cache.clone(), w.v_cache.clone()
    k0[int(bt[0, 5])] = 0
    v0[int(bt[0, 5])] = 0
    for window, tables, k, v, bits in ((0, bad, k0, v0, 1), (60, bad, k0, v0, 1),
                                       (60, skipped, w.k_cache, w.v_cache, 0)):
        out, status = with_checks(w.num_blocks, lambda: pa.paged_attn_decode_mods(
            w.q, w.k_cache, w.v_cache, tables, w.seq_lens, w.scale, window=window))
        assert status == bits
        within(out, serving.attend(f64(w.q), f64(k), f64(v), None, bt, lens, scale, window=window))
        out, status = with_checks(w.num_blocks, lambda: pa.paged_attn_decode_multi_mods(
            q, w.k_cache, w.v_cache, i32(qo), tables, w.seq_lens, w.scale, window=window))
        assert status == bits
        within(out, serving.attend(f64(q), f64(k), f64(v), qo, bt, lens, scale, window=window))
    # a prefix's page
    out, status = with_checks(w.num_blocks, lambda: pa.paged_attn_decode_shared(
        w.q[1:].contiguous(), w.k_cache, w.v_cache, i32([0, 1]), bad[:1].clone(), i32([100]),
        w.block_tables[1:].clone(), i32([40]), w.scale))
    assert status == 1
    within(out, serving.attend_shared(f64(w.q[1:]), f64(k0), f64(v0), [0, 1], bt[:1], [100], bt[1:],
                                      [40], scale))


def test_a_bad_fp8_page_is_a_page_of_zeros():
    lens = [100, 40]
    w = workloads.make(workloads.custom_spec("bad8", 2, 8, 2, 128, 16, lens), device="cuda")
    f = workloads.to_fp8(w)
    bt = w.block_tables.cpu().numpy()
    bad = w.block_tables.clone()
    bad[0, 5] = w.num_blocks + 3
    out, status = with_checks(w.num_blocks, lambda: pa.paged_attn_decode_fp8_mods(
        w.q, f.k8, f.v8, f.k_scale, f.v_scale, bad, w.seq_lens, w.scale))
    assert status == 1
    k = f.k8.view(torch.float8_e4m3fn).double() * f.k_scale.double()[..., None]
    v = f.v8.view(torch.float8_e4m3fn).double() * f.v_scale.double()[..., None]
    k[int(bt[0, 5])] = 0
    v[int(bt[0, 5])] = 0
    within(out, serving.attend(f64(w.q), k.cpu().numpy(), v.cpu().numpy(), None, bt, lens,
                               float(np.float32(w.scale)), eps_p=serving.F16_STEP, f16=True))
