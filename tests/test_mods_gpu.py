"""Decode with score options against the float64 definition, element by element within
the bound that the roundings allow (oracle.serving), over bf16 and FP8 caches, head
dims, page sizes and group sizes, with NaN in every row that no query sees."""
import math

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


def poison_unseen(w, lens, seen_of):
    """NaN into the rows no query sees (in pages that another of their rows shares
    too), and into the table entries of pages without a seen row a spare block."""
    BS = w.spec.block_size
    bt = w.block_tables.cpu().numpy()
    kc, vc = w.k_cache, w.v_cache
    for s, n in enumerate(lens):
        seen = seen_of(s, n)
        hidden = np.nonzero(~seen)[0]
        for t in hidden:
            b = int(bt[s, t // BS])
            kc[b, :, t % BS] = float("nan")
            vc[b, :, t % BS] = float("nan")
        for page in range(-(-n // BS)):
            if not seen[page * BS:(page + 1) * BS].any():
                bt[s, page] = w.poison_block
    w.block_tables.copy_(torch.tensor(bt))


def slopes_of(H):
    return np.array([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=np.float32)


def case(lens, H_q, H_kv, D, BS, seed, softcap=0.0, alibi=False, window=0, prefix=None, docs=None,
         q_gain=1.0, max_len=None):
    sp = workloads.custom_spec("mods", len(lens), H_q, H_kv, D, BS, lens, max_len=max_len)
    w = workloads.make(sp, seed=seed, device="cuda", poison="nan")
    w.q.mul_(q_gain)
    prefix = None if prefix is None else np.asarray(prefix)
    docs = None if docs is None else np.asarray(docs)

    def seen_of(s, n):
        return serving.visible(np.array([n - 1]), n, True, window,
                               0 if prefix is None else int(prefix[s]),
                               None if docs is None else docs[s:s + 1])[0]

    poison_unseen(w, lens, seen_of)
    kw = dict(softcap=softcap, alibi_slopes=torch.tensor(slopes_of(H_q)).cuda() if alibi else None,
              window=window, prefix_lens=None if prefix is None else i32(prefix),
              doc_starts=None if docs is None else i32(docs))
    okw = dict(softcap=softcap, slopes=slopes_of(H_q).astype(np.float64) if alibi else None,
               window=window, prefix_lens=prefix, doc_starts=docs)
    return w, kw, okw


def within(out, res, what=""):
    got = serving.bf16_to_f64(out)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    err = np.abs(got - res.out)  # (a row that sees nothing has no error and no bound)
    over = np.divide(err, res.tol, out=np.where(err > 0, np.inf, 0.0), where=res.tol > 0)
    assert over.max() <= 1.0, f"{what}: {over.max():.3f} of the bound at {np.unravel_index(over.argmax(), over.shape)}"


def check_bf16(w, kw, okw, what=""):
    out = pa.paged_attn_decode_mods(w.q, w.k_cache, w.v_cache, w.block_tables, w.seq_lens, w.scale,
                                    **kw)
    torch.cuda.synchronize()
    res = serving.attend(serving.bf16_to_f64(w.q), serving.bf16_to_f64(w.k_cache),
                         serving.bf16_to_f64(w.v_cache), None, w.block_tables.cpu().numpy(),
                         w.lens_list, float(np.float32(w.scale)), **okw)
    within(out, res, what)
    return out


def check_fp8(w, kw, okw, what=""):
    f = workloads.to_fp8(w)
    # rows nobody sees: the e4m3 NaN byte and NaN floats
    nan = torch.isnan(w.k_cache).any(-1)
    for c, sc in ((f.k8, f.k_scale), (f.v8, f.v_scale)):
        c[nan] = 0x7F
        sc[nan] = float("nan")
    out = pa.paged_attn_decode_fp8_mods(f.q, f.k8, f.v8, f.k_scale, f.v_scale, f.block_tables,
                                        f.seq_lens, f.scale, **kw)
    torch.cuda.synchronize()
    deq = [c.view(torch.float8_e4m3fn).cpu().float().numpy().astype(np.float64) *
           sc.cpu().numpy().astype(np.float64)[..., None] for c, sc in ((f.k8, f.k_scale),
                                                                       (f.v8, f.v_scale))]
    res = serving.attend(serving.bf16_to_f64(f.q), *deq, None, f.block_tables.cpu().numpy(),
                         w.lens_list, float(np.float32(w.scale)), eps_p=serving.F16_STEP, f16=True,
                         **okw)
    within(out, res, what)


LENS = [1, 15, 16, 17, 31, 33, 64, 100, 257, 0, 1000, 2]

OPTIONS = [
    dict(softcap=30.0), dict(softcap=0.5), dict(alibi=True), dict(window=1), dict(window=16),
    dict(window=37), dict(window=5000), dict(prefix=[3] * 12),
    dict(window=40, prefix=[4, 4, 20, 0, 9, 40, 1, 33, 16, 7, 90, 5]),
    dict(docs=[0, 14, 15, 16, 31, 5, 63, 90, 16, 3, 999, 1]),
    dict(softcap=50.0, alibi=True, window=50, prefix=[2, 0, 3, 16, 17, 5, 6, 7, 100, 9, 32, 1],
         docs=[0, 3, 16, 2, 20, 32, 10, 80, 250, 0, 980, 0]),
]


@pytest.mark.parametrize("D,BS,H_q,H_kv", [(64, 16, 4, 2), (64, 32, 16, 1), (128, 16, 8, 2),
                                           (128, 32, 6, 1), (256, 16, 12, 2), (256, 32, 16, 1),
                                           (128, 16, 16, 1), (256, 16, 2, 2)])
@pytest.mark.parametrize("o", range(len(OPTIONS)))
def test_options(D, BS, H_q, H_kv, o):
    w, kw, okw = case(LENS, H_q, H_kv, D, BS, 17 * D + o, q_gain=3.0, **OPTIONS[o])
    check_bf16(w, kw, okw, f"bf16 {OPTIONS[o]}")
    if D >= 128:
        check_fp8(w, kw, okw, f"fp8 {OPTIONS[o]}")


@pytest.mark.parametrize("name", ["tiny", "llama8b"])
@pytest.mark.parametrize("cap,window", [(50.0, 0), (30.0, 300)])
def test_workload_shapes(name, cap, window):
    sp = workloads.spec(name)
    lens = [int(x) for x in workloads.make(name, device="cpu").seq_lens][:6] if name == "tiny" else \
        [4096, 513, 1029, 2048, 3999, 700]
    w, kw, okw = case(lens, sp.H_q, sp.H_kv, sp.D, sp.block_size, 3, softcap=cap, window=window,
                      alibi=window > 0, prefix=[4] * len(lens))
    check_bf16(w, kw, okw, name)


def test_a_sequence_split_over_all_ctas_with_a_hole():
    """One long sequence: a prefix, a gap of skipped pages, a window that ends inside pages."""
    w, kw, okw = case([50021, 900], 8, 1, 128, 16, 5, window=20011, prefix=[3333, 10], alibi=True,
                      softcap=20.0)
    check_bf16(w, kw, okw)
    check_fp8(w, kw, okw)


def test_no_options_equal_the_plain_decode():
    w = workloads.make("llama8b", device="cuda", poison="nan")
    a = pa.paged_attn_decode(w.q, w.k_cache, w.v_cache, w.block_tables, w.seq_lens, w.scale)
    b = pa.paged_attn_decode_mods(w.q, w.k_cache, w.v_cache, w.block_tables, w.seq_lens, w.scale)
    f = workloads.to_fp8(w)
    args = (f.q, f.k8, f.v8, f.k_scale, f.v_scale, f.block_tables, f.seq_lens, f.scale)
    c, d = pa.paged_attn_decode_fp8(*args), pa.paged_attn_decode_fp8_mods(*args)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    # (the FP8 scores take their two factors in another order)
    assert (c.float() - d.float()).abs().max() <= 2.0 ** -8 * c.float().abs().max()


def test_queries_that_see_nothing_are_zero():
    """A document that begins past the query; a clamp of values outside [0, L]."""
    w, kw, okw = case([40, 17, 100], 4, 2, 64, 16, 6, docs=[40, 500, -3], prefix=[0, -5, 1000])
    out = check_bf16(w, kw, okw)
    assert torch.count_nonzero(out[:2]) == 0 and torch.count_nonzero(out[2]) > 0


@pytest.mark.parametrize("cap", [1e-3, 1.0, 1e6])
@pytest.mark.parametrize("gain", [0.01, 1.0, 60.0])
def test_caps_and_scores_of_any_size(cap, gain):
    w, kw, okw = case([300, 77], 8, 2, 128, 16, 8, softcap=cap, q_gain=gain)
    check_bf16(w, kw, okw, f"cap {cap} gain {gain}")


def test_a_very_long_sequence_has_a_hole_past_any_int16():
    w, kw, okw = case([120007], 2, 1, 64, 32, 9, window=77, prefix=[65])
    check_bf16(w, kw, okw)


def test_more_sequences_than_one_launch_holds():
    lens = list(np.random.default_rng(12).integers(0, 60, size=4500))
    pre, docs = [s % 3 for s in range(4500)], [s % 29 for s in range(4500)]
    w, kw, okw = case(lens, 4, 1, 64, 16, 13, window=20, prefix=pre, docs=docs, max_len=64)
    check_bf16(w, kw, okw)


def test_repeat_calls_are_bitwise_identical_and_share_a_workspace():
    w, kw, _ = case([4000, 100, 2222], 32, 8, 128, 16, 14, softcap=30.0, window=1500)
    n = pa.paged_attn_mods_workspace_bytes(3, 32, 8, 128, w.max_blocks_per_seq, 16)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    args = (w.q, w.k_cache, w.v_cache, w.block_tables, w.seq_lens, w.scale)
    a = pa.paged_attn_decode_mods(*args, **kw)
    b = pa.paged_attn_decode_mods(*args, workspace=ws, **kw)
    c = pa.paged_attn_decode_mods(*args, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(b, c)
    with pytest.raises(pa.PagedAttnError, match="workspace"):
        pa.paged_attn_decode_mods(*args, workspace=ws[256:512], **kw)


def test_a_capture_brings_its_workspace():
    w, kw, okw = case([4000, 100, 2222], 32, 8, 128, 16, 15, softcap=30.0, window=1500)
    args = (w.q, w.k_cache, w.v_cache, w.block_tables, w.seq_lens, w.scale)
    eager = check_bf16(w, kw, okw)
    out = torch.zeros_like(w.q)
    n = pa.paged_attn_mods_workspace_bytes(3, 32, 8, 128, w.max_blocks_per_seq, 16)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(pa.PagedAttnError, match="workspace"):
            pa.paged_attn_decode_mods(*args, out=out, **kw)
        pa.paged_attn_decode_mods(*args, out=out, workspace=ws, **kw)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_bad_pages_are_reported_and_read_as_zeros():
    w, kw, okw = case([100, 40], 8, 2, 128, 16, 16, window=60)
    status = i32([0])
    bt = w.block_tables.clone()
    bt[0, 5] = w.num_blocks + 3
    try:
        pa.paged_attn_set_checks(w.num_blocks, status)
        bt2 = w.block_tables.clone()
        bt2[0, 0] = -9                      # a skipped page's entry is not looked at
        pa.paged_attn_decode_mods(w.q, w.k_cache, w.v_cache, bt2, w.seq_lens, w.scale, **kw)
        torch.cuda.synchronize()
        assert int(status) == 0
        pa.paged_attn_decode_mods(w.q, w.k_cache, w.v_cache, bt, w.seq_lens, w.scale, **kw)
        torch.cuda.synchronize()
        assert int(status) == 1
    finally:
        pa.paged_attn_set_checks(0, None)
