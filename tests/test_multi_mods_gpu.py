"""Attention of many query tokens per sequence with score options against the float64
definition, element by element within the bound that the roundings allow, with
NaN in every cache row that no query of its sequence sees."""
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


def slopes_of(H):
    return np.array([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=np.float32)


def within(out, res, what=""):
    got = serving.bf16_to_f64(out)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    err = np.abs(got - res.out)
    over = np.divide(err, res.tol, out=np.where(err > 0, np.inf, 0.0), where=res.tol > 0)
    at = np.unravel_index(over.argmax(), over.shape)
    assert over.max() <= 1.0, f"{what}: {over.max():.3f} of the bound at {at}"


def run_case(lens, qlens, H_q, H_kv, D, BS, seed, causal=True, softcap=0.0, alibi=False, window=0,
             prefix=None, doc=0, gain=1.0, max_len=None, scale=None, workspace=None):
    """doc: sequences are packed from documents of that many tokens."""
    kw = {} if scale is None else dict(scale=scale)
    sp = workloads.custom_spec("mm", len(lens), H_q, H_kv, D, BS, lens, max_len=max_len, **kw)
    w = workloads.make(sp, seed=seed, device="cuda", poison="nan")
    g = torch.Generator().manual_seed(seed)
    qo = np.concatenate([[0], np.cumsum(qlens)])
    q = (torch.randn(int(qo[-1]), H_q, D, generator=g) * gain).to(torch.bfloat16).cuda()
    prefix = None if prefix is None else np.resize(np.asarray(prefix), len(lens))
    docs = None
    if doc:
        docs = np.concatenate([np.maximum(0, n - m + np.arange(m)) // doc * doc
                               for n, m in zip(lens, qlens)] + [np.zeros(0, dtype=int)]).astype(int)
    bt = w.block_tables.cpu().numpy()
    for s, (n, m) in enumerate(zip(lens, qlens)):
        pos = n - m + np.arange(m)
        seen = serving.visible(pos, n, causal, window, 0 if prefix is None else int(prefix[s]),
                               None if docs is None else docs[qo[s]:qo[s + 1]])
        for t in np.nonzero(~seen.any(axis=0))[0] if m else range(n):
            for c in (w.k_cache, w.v_cache):
                c[int(bt[s, t // BS]), :, t % BS] = float("nan")
    slopes = slopes_of(H_q)
    out = torch.full_like(q, 7.0)
    pa.paged_attn_decode_multi_mods(
        q, w.k_cache, w.v_cache, i32(qo), w.block_tables, w.seq_lens, w.scale, causal=causal,
        softcap=softcap, alibi_slopes=torch.tensor(slopes).cuda() if alibi else None,
        window=window, prefix_lens=None if prefix is None else i32(prefix),
        doc_starts=None if docs is None else i32(docs), out=out, workspace=workspace)
    torch.cuda.synchronize()
    res = serving.attend(serving.bf16_to_f64(q), serving.bf16_to_f64(w.k_cache),
                         serving.bf16_to_f64(w.v_cache), qo, bt, lens, float(np.float32(w.scale)),
                         causal=causal, softcap=softcap,
                         slopes=slopes.astype(np.float64) if alibi else None, window=window,
                         prefix_lens=prefix, doc_starts=docs)
    within(out, res, f"D{D} BS{BS} G{H_q // H_kv}")
    return out


# one tile of keys and one of rows, and every way to leave them
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("BS", [16, 32])
def test_one_sequence_one_tile(D, BS):
    run_case([64], [64], 1, 1, D, BS, 1, causal=False)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("BS", [16, 32])
@pytest.mark.parametrize("n,m,G", [(1, 1, 1), (17, 3, 4), (128, 128, 1), (129, 129, 1),
                                   (130, 33, 4), (257, 64, 4), (300, 300, 1), (511, 43, 6),
                                   (640, 40, 16)])
def test_row_and_token_tiles(D, BS, n, m, G):
    run_case([n], [m], 2 * G, 2, D, BS, n + m)


LENS = [1, 15, 16, 17, 33, 100, 257, 0, 700, 64, 129, 40]
QLENS = [1, 3, 16, 0, 33, 70, 130, 0, 300, 64, 129, 7]

OPTIONS = [
    dict(causal=False), dict(softcap=30.0), dict(softcap=0.5, causal=False), dict(alibi=True),
    dict(alibi=True, causal=False), dict(window=1), dict(window=16), dict(window=150),
    dict(window=64, causal=False), dict(prefix=[3, 140, 0]), dict(doc=50), dict(doc=128),
    dict(doc=97, causal=False),
    dict(softcap=50.0, alibi=True, window=45, prefix=[0, 5, 33, 200], doc=60),
]


@pytest.mark.parametrize("D,BS,H_q,H_kv", [(64, 16, 4, 2), (128, 16, 4, 1), (128, 32, 6, 2),
                                           (256, 16, 6, 1), (256, 32, 2, 2), (64, 32, 16, 1)])
@pytest.mark.parametrize("o", range(len(OPTIONS)))
def test_options(D, BS, H_q, H_kv, o):
    run_case(LENS, QLENS, H_q, H_kv, D, BS, 31 * D + o, gain=2.0, **OPTIONS[o])


def test_more_queries_than_tokens_and_unowned_rows():
    """q_len > L: the first rows see no token (zero); rows past the last sequence stay."""
    out = run_case([3, 40, 0, 17], [5, 60, 4, 1], 8, 2, 128, 16, 3)
    assert torch.count_nonzero(out[:2]) == 0 and torch.count_nonzero(out[65:69]) == 0
    w = workloads.make(workloads.custom_spec("own", 1, 4, 2, 64, 16, [40]), device="cuda")
    q = torch.randn(9, 4, 64, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 3.0)
    pa.paged_attn_decode_multi_mods(q, w.k_cache, w.v_cache, i32([0, 5]), w.block_tables,
                                    w.seq_lens, w.scale, out=out)
    assert (out[5:] == 3.0).all() and not (out[:5] == 3.0).all()


def test_a_long_sequence_is_split_and_merged():
    run_case([9001], [5], 8, 1, 128, 16, 4, softcap=20.0)
    run_case([9001, 30], [3, 30], 4, 1, 256, 32, 5, window=4000, prefix=[1111, 7])
    run_case([5003], [2], 2, 1, 64, 16, 6, alibi=True)


def test_many_short_sequences():
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 90, size=700)
    qlens = np.minimum(rng.integers(0, 12, size=700), lens)
    run_case(list(lens), list(qlens), 4, 1, 64, 16, 8, max_len=96)


def test_peaked_scores_rescale():
    """Scores that grow along the sequence raise the running maximum again and again."""
    run_case([900], [200], 4, 2, 128, 16, 9, gain=40.0)
    run_case([900], [200], 4, 2, 256, 16, 10, gain=40.0)
    run_case([600], [50], 4, 2, 128, 16, 11, gain=60.0, softcap=1e6)


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-20, 3.0])
def test_scales(scale):
    run_case([300, 20], [140, 20], 2, 1, 128, 16, 12, scale=scale)
    run_case([300, 20], [140, 20], 2, 1, 128, 16, 13, scale=scale, softcap=5.0, window=100)


def test_equals_the_plain_multi_token_decode():
    w = workloads.make("llama8b", device="cuda", poison="nan")
    qo = i32(np.arange(33) * 4)
    q = torch.randn(128, 32, 128, device="cuda").to(torch.bfloat16)
    a = pa.paged_attn_decode_multi(q, w.k_cache, w.v_cache, qo, w.block_tables, w.seq_lens,
                                   w.scale, 4)
    b = pa.paged_attn_decode_multi_mods(q, w.k_cache, w.v_cache, qo, w.block_tables, w.seq_lens,
                                        w.scale)
    # each is within (2 eps + eps) of the values' mean magnitude (below 1 here) plus 1e-4
    assert (a.float() - b.float()).abs().max() <= 6 * 2.0 ** -8 + 2e-4


def test_repeat_calls_and_a_captured_one_are_bitwise_identical():
    w = workloads.make(workloads.custom_spec("rep", 2, 8, 2, 128, 16, [3000, 500]), device="cuda")
    q = torch.randn(20, 8, 128, device="cuda").to(torch.bfloat16)
    args = (q, w.k_cache, w.v_cache, i32([0, 12, 20]), w.block_tables, w.seq_lens, w.scale)
    kw = dict(softcap=30.0, window=2000)
    a = pa.paged_attn_decode_multi_mods(*args, **kw)
    b = pa.paged_attn_decode_multi_mods(*args, **kw)
    assert torch.equal(a, b)
    n = pa.paged_attn_multi_mods_workspace_bytes(2, 20, 8, 2, 128, w.max_blocks_per_seq, 16)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(pa.PagedAttnError, match="workspace"):
            pa.paged_attn_decode_multi_mods(*args, **kw, out=out)
        pa.paged_attn_decode_multi_mods(*args, **kw, out=out, workspace=ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a)
    with pytest.raises(pa.PagedAttnError, match="workspace"):
        pa.paged_attn_decode_multi_mods(*args, **kw, workspace=ws[:256])


def test_bad_pages_are_reported():
    w = workloads.make(workloads.custom_spec("bad", 1, 8, 2, 128, 16, [500]), device="cuda")
    q = torch.randn(20, 8, 128, device="cuda").to(torch.bfloat16)
    status = i32([0])
    try:
        pa.paged_attn_set_checks(w.num_blocks, status)
        for entry, bits in ((0, 0), (31, 1)):
            bt = w.block_tables.clone()
            if bits:
                bt[0, entry] = w.num_blocks
            pa.paged_attn_decode_multi_mods(q, w.k_cache, w.v_cache, i32([0, 20]), bt, w.seq_lens,
                                            w.scale)
            torch.cuda.synchronize()
            assert int(status) == bits
        status.zero_()
        pa.paged_attn_decode_multi_mods(q, w.k_cache, w.v_cache, i32([0, 20]), w.block_tables,
                                        i32([5000]), w.scale)
        torch.cuda.synchronize()
        assert int(status) & 2
    finally:
        pa.paged_attn_set_checks(0, None)


# Launches with as many pieces as the GPU has places run the kernel of two teams (head_dim 64
# and 128): on both row tiles of a full piece, on alternate token tiles of a short one.
@pytest.mark.parametrize("D,BS", [(64, 32), (128, 16)])
@pytest.mark.parametrize("o", range(len(OPTIONS)))
def test_options_on_many_pieces(D, BS, o):
    run_case(LENS, QLENS, 32, 8, D, BS, 17 * D + BS + o, gain=2.0, **OPTIONS[o])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 1.0, 1e6])
@pytest.mark.parametrize("gain", [0.01, 60.0])
def test_caps_and_scores_of_any_size_on_many_pieces(D, cap, gain):
    run_case([300, 400, 129], [300, 257, 70], 32, 32, D, 16, 14, softcap=cap, gain=gain)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("cap", [1e-3, 1.0, 1e6])
@pytest.mark.parametrize("gain", [0.01, 60.0])
def test_caps_and_scores_of_any_size(D, cap, gain, alibi):
    run_case([300, 77], [130, 77], 4, 2, D, 16, 15, softcap=cap, gain=gain, alibi=alibi)


def test_repeat_calls_on_many_pieces_are_bitwise_identical():
    a = run_case([1500, 700], [900, 700], 32, 8, 128, 16, 16, softcap=50.0, window=333)
    for _ in range(3):
        b = run_case([1500, 700], [900, 700], 32, 8, 128, 16, 16, softcap=50.0, window=333)
        assert torch.equal(a, b)
