"""Refusals of the serving entry points, on the host: no CUDA call is made."""
import pytest
import torch

import paged_kv_gqa_decode_gb300 as pa
from paged_kv_gqa_decode_gb300 import build as pbuild

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.load()


MODS = dict(q=16, k=16, v=16, out=16, bt=16, sl=16, num_seqs=2, H_q=8, H_kv=2, D=128, maxb=4,
            BS=16, scale=0.125, softcap=0.0, slopes=None, window=0, prefix=None, docs=None,
            ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(H_q=6, H_kv=4), -2), (dict(H_q=34, H_kv=2), -2), (dict(D=96), -3), (dict(BS=8), -4),
    (dict(num_seqs=-1), -5), (dict(maxb=0), -5), (dict(scale=float("inf")), -8),
    (dict(q=None), -1), (dict(out=24), -1), (dict(softcap=-1.0), -11),
    (dict(softcap=float("nan")), -11), (dict(softcap=float("inf")), -11), (dict(window=-1), -11),
    (dict(slopes=2), -1), (dict(prefix=6), -1), (dict(docs=17), -1),
])
def test_decode_mods_refuses(lib, kw, code):
    a = dict(MODS, **kw)
    assert lib.paged_attn_decode_mods(*a.values()) == code
    f = {}
    for name, x in a.items():
        f[name] = x
        if name == "v":
            f.update(ks=16, vs=16)
    assert lib.paged_attn_decode_fp8_mods(*f.values()) == code


def test_fp8_mods_refuses_head_dim_64_and_null_floats(lib):
    a = dict(MODS)
    base = list(a.values())
    for D, ks, code in ((64, 16, -3), (128, None, -1), (128, 24, -1)):
        args = base[:3] + [ks, 16] + base[3:]
        args[11] = D
        assert lib.paged_attn_decode_fp8_mods(*args) == code


def test_empty_batches(lib):
    a = dict(MODS, num_seqs=0, q=None, k=None, v=None, out=None, bt=None, sl=None)
    assert lib.paged_attn_decode_mods(*a.values()) == 0
    # (not the assignment: its padding slots and counts are written whatever comes)
    assert lib.paged_kv_assign(*[None] * 10, 0, 4, 16, 10, 10, None) == -1
    assert lib.paged_kv_append_slots(None, None, 256, 256, None, None, None, 0, 2, 128, 16, 5,
                                     None) == 0


ASSIGN = dict(lens=16, new=16, bt=16, free=16, count=4, lens_out=16, qo=16, slots=16, left=4,
              refused=None, num_seqs=2, maxb=4, BS=16, cap=8, max_new=8, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(BS=8), -4), (dict(maxb=0), -5), (dict(num_seqs=-1), -5), (dict(cap=-1), -5),
    (dict(max_new=-1), -5), (dict(lens=None), -1), (dict(new=8), -1), (dict(bt=None), -1),
    (dict(free=None), -1), (dict(count=None), -1), (dict(count=2), -1), (dict(left=None), -1),
    (dict(qo=None), -1), (dict(slots=24), -1), (dict(refused=2), -1), (dict(lens_out=None), -1),
])
def test_assign_refuses(lib, kw, code):
    assert lib.paged_kv_assign(*dict(ASSIGN, **kw).values()) == code


SLOTS = dict(k=16, v=16, ks=256, vs=256, kc=16, vc=16, slots=16, rows=3, H_kv=2, D=128, BS=16,
             nb=5, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(H_kv=0), -2), (dict(D=96), -3), (dict(BS=64), -4), (dict(rows=-1), -5), (dict(nb=0), -5),
    (dict(nb=2 ** 31), -5), (dict(ks=248), -5), (dict(vs=260), -5), (dict(k=8), -1),
    (dict(vc=None), -1), (dict(slots=None), -1),
])
def test_append_slots_refuses(lib, kw, code):
    assert lib.paged_kv_append_slots(*dict(SLOTS, **kw).values()) == code


def problem():
    q = torch.zeros(3, 8, 128, dtype=BF)
    kc = torch.zeros(10, 2, 16, 128, dtype=BF)
    bt = torch.zeros(3, 4, dtype=torch.int32)
    return q, kc, kc.clone(), bt, torch.ones(3, dtype=torch.int32)


@pytest.mark.parametrize("kw", [
    dict(alibi_slopes=torch.zeros(4)), dict(alibi_slopes=torch.zeros(8, dtype=torch.float64)),
    dict(prefix_lens=torch.zeros(3, dtype=torch.int64)),
    dict(doc_starts=torch.zeros(4, dtype=torch.int32)), dict(out=torch.zeros(3, 8, 64, dtype=BF)),
    dict(out=torch.zeros(3, 8, 128)),
])
def test_the_binding_refuses_other_shapes_and_types(kw):
    with pytest.raises(ValueError):
        pa.paged_attn_decode_mods(*problem(), 0.1, **kw)


def test_the_binding_refuses_mismatched_problems():
    q, kc, vc, bt, sl = problem()
    for bad in ((q.float(), kc, vc, bt, sl), (q[:2], kc, vc, bt, sl),
                (q, kc[..., :64].contiguous(), vc, bt, sl), (q, kc, vc, bt.long(), sl),
                (q, kc, vc, bt, sl.long()), (q, kc.transpose(0, 1), vc, bt, sl),
                (q, kc, vc[:5], bt, sl)):
        with pytest.raises(ValueError):
            pa.paged_attn_decode_mods(*bad, 0.1)


def test_the_binding_refuses_unpinned_host_tensors():
    with pytest.raises(ValueError, match="pinned"):
        pa.paged_attn_decode_mods(*problem(), 0.1)


def test_the_binding_refuses_scattered_new_rows():
    _, kc, vc, _, _ = problem()
    slots = torch.zeros(3, dtype=torch.int64)
    good = torch.zeros(3, 2, 128, dtype=BF)
    for bad in (good.float(), torch.zeros(3, 128, 2, dtype=BF).transpose(1, 2),
                torch.zeros(3, 4, 128, dtype=BF)[:, ::2], torch.zeros(3, 2, 64, dtype=BF)):
        with pytest.raises(ValueError):
            pa.paged_kv_append_slots(bad, good, kc, vc, slots)
    with pytest.raises(ValueError):
        pa.paged_kv_append_slots(good, good, kc, vc, slots.int())


MULTI = dict(q=16, k=16, v=16, out=16, qo=16, bt=16, sl=16, num_seqs=2, total_q=5, H_q=8, H_kv=2,
             D=128, maxb=4, BS=16, scale=0.125, causal=1, softcap=0.0, slopes=None, window=0,
             prefix=None, docs=None, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(H_q=6, H_kv=4), -2), (dict(D=32), -3), (dict(BS=64), -4), (dict(num_seqs=-1), -5),
    (dict(total_q=-1), -5), (dict(total_q=2 ** 29), -5), (dict(scale=float("nan")), -8),
    (dict(q=8), -1), (dict(qo=None), -1), (dict(softcap=1e-31), -11), (dict(softcap=2e30), -11),
    (dict(softcap=1e-25, scale=1e6), -11), (dict(window=-5), -11), (dict(docs=1), -1),
    (dict(maxb=2 ** 27 - 8), -5),
])
def test_decode_multi_mods_refuses(lib, kw, code):
    assert lib.paged_attn_decode_multi_mods(*dict(MULTI, **kw).values()) == code


def test_empty_query_batches_are_no_ops(lib):
    for kw in (dict(total_q=0), dict(num_seqs=0)):
        a = dict(MULTI, q=None, k=None, v=None, out=None, qo=None, bt=None, sl=None, **kw)
        assert lib.paged_attn_decode_multi_mods(*a.values()) == 0


SHARED = dict(q=16, k=16, v=16, out=16, gi=16, pt=16, pl=16, groups=1, pmax=4, bt=16, sl=16,
              num_seqs=2, H_q=8, H_kv=2, D=128, maxb=4, BS=16, scale=0.125, softcap=0.0,
              slopes=None, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(H_q=6, H_kv=4), -2), (dict(D=32), -3), (dict(BS=64), -4), (dict(num_seqs=-1), -5),
    (dict(groups=-1), -5), (dict(pmax=0), -5), (dict(pmax=2 ** 27 - 8), -5),
    (dict(scale=float("inf")), -8), (dict(gi=None), -1), (dict(pt=8), -1), (dict(pl=None), -1),
    (dict(bt=None), -1), (dict(softcap=-2.0), -11), (dict(slopes=3), -1),
])
def test_decode_shared_refuses(lib, kw, code):
    assert lib.paged_attn_decode_shared(*dict(SHARED, **kw).values()) == code


@pytest.mark.parametrize("name,args", [
    ("paged_attn_mods_workspace_bytes", (4, 6, 4, 128, 8, 16)),
    ("paged_attn_mods_workspace_bytes", (4, 8, 2, 80, 8, 16)),
    ("paged_attn_multi_mods_workspace_bytes", (4, -1, 8, 2, 128, 8, 16)),
    ("paged_attn_multi_mods_workspace_bytes", (4, 5, 8, 2, 128, 8, 8)),
    ("paged_attn_shared_workspace_bytes", (4, -1, 8, 2, 128, 8, 16)),
])
def test_workspace_queries_reject_bad_sizes(lib, name, args):
    assert getattr(lib, name)(*args) == 0


def test_the_binding_refuses_mismatched_groups_and_offsets():
    q, kc, vc, bt, sl = problem()
    gi, pt, pl = (torch.zeros(2, dtype=torch.int32), torch.zeros(1, 4, dtype=torch.int32),
                  torch.zeros(1, dtype=torch.int32))
    for bad in ((gi[:1], pt, pl), (gi, pt[0], pl), (gi, pt, gi), (gi.long(), pt, pl)):
        with pytest.raises(ValueError):
            pa.paged_attn_decode_shared(q, kc, vc, *bad, bt, sl, 0.1)
    for qo in (torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)):
        with pytest.raises(ValueError):
            pa.paged_attn_decode_multi_mods(q, kc, vc, qo, bt, sl, 0.1)
