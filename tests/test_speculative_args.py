"""Refusals of the entry points for trees, rotation and page handling, on the host: no CUDA
call is made."""
import pytest
import torch

import paged_kv_gqa_decode_gb300 as pa
from paged_kv_gqa_decode_gb300 import build as pbuild

BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def lib():
    pbuild.build()
    return pa.load()


TREE = dict(q=16, k=16, v=16, out=16, qo=16, mask=16, words=2, bt=16, sl=16, num_seqs=2, total_q=5,
            H_q=8, H_kv=2, D=128, maxb=4, BS=16, scale=0.125, softcap=0.0, slopes=None, window=0,
            prefix=None, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(H_q=6, H_kv=4), -2), (dict(D=32), -3), (dict(BS=64), -4), (dict(num_seqs=-1), -5),
    (dict(total_q=-1), -5), (dict(total_q=2 ** 29), -5), (dict(words=0), -5), (dict(words=9), -5),
    (dict(scale=float("nan")), -8), (dict(q=8), -1), (dict(qo=None), -1), (dict(mask=None), -1),
    (dict(mask=24), -1), (dict(softcap=-1.0), -11), (dict(window=-5), -11), (dict(prefix=1), -1),
    (dict(slopes=2), -1), (dict(maxb=2 ** 27 - 8), -5),
])
def test_tree_refuses(lib, kw, code):
    assert lib.paged_attn_decode_tree(*dict(TREE, **kw).values()) == code


ROPE = dict(q=16, k=16, v=16, qs=1024, ks=256, vs=256, out=32, kc=16, vc=16, kf=None, vf=None,
            slots=16, pos=16, axes=1, axis=None, cs=16, most=100, rot=64, inter=0, qn=None, kn=None,
            eps=1e-6, rows=3, H_q=8, H_kv=2, D=128, BS=16, nb=5, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(H_q=6, H_kv=4), -2), (dict(D=96), -3), (dict(BS=64), -4), (dict(rows=-1), -5),
    (dict(nb=0), -5), (dict(nb=2 ** 31), -5), (dict(qs=1016), -5), (dict(ks=248), -5),
    (dict(vs=260), -5), (dict(rot=8), -12), (dict(rot=144), -12), (dict(rot=-16), -12),
    (dict(axes=0), -12), (dict(most=0), -12), (dict(eps=-1.0), -12), (dict(eps=float("nan")), -12),
    (dict(eps=float("inf")), -12), (dict(q=8), -1), (dict(out=None), -1), (dict(kc=None), -1),
    (dict(slots=None), -1), (dict(pos=None), -1), (dict(cs=None), -1), (dict(cs=24), -1),
    (dict(axis=8), -1), (dict(qn=8), -1), (dict(kn=4), -1), (dict(kf=16), -1), (dict(vf=16), -1),
    (dict(kf=16, vf=24), -1), (dict(kf=16, vf=16, D=64, qs=512, ks=128, vs=128), -3),
    (dict(out=16, qs=1032), -1),
])
def test_rope_append_refuses(lib, kw, code):
    assert lib.paged_kv_rope_append_slots(*dict(ROPE, **kw).values()) == code


# q at 2^20, three rows of 2048 bytes 8192 apart; k and v far from it, rows of 512 bytes 1024 apart
APART = dict(ROPE, q=2 ** 20, qs=4096, k=2 ** 24, ks=512, v=2 ** 25, vs=512, pos=2 ** 10, slots=2 ** 10)


@pytest.mark.parametrize("out", [
    2 ** 20 - 6144 + 16, 2 ** 20, 2 ** 20 + 16, 2 ** 20 + 2032, 2 ** 20 + 2064, 2 ** 20 + 2 * 8192 + 2032,
    2 ** 24 - 6144 + 16, 2 ** 24, 2 ** 24 + 2 * 1024 + 496, 2 ** 25 - 16, 2 ** 25 + 512, 2 ** 25 + 2 * 1024 + 496,
])
def test_rope_append_refuses_queries_out_over_its_inputs(lib, out):
    """3 rows of 2048 bytes in one: from the last place before an input to the last one in it."""
    assert lib.paged_kv_rope_append_slots(*dict(APART, out=out).values()) == -1


COMPACT = dict(kc=16, vc=16, kf=None, vf=None, qo=16, acc=16, bt=16, sl=16, out=32, n=2, most=4,
               H_kv=2, D=128, maxb=4, BS=16, nb=5, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(H_kv=0), -2), (dict(D=96), -3), (dict(BS=64), -4), (dict(n=-1), -5), (dict(maxb=0), -5),
    (dict(most=-1), -5), (dict(most=2 ** 30 + 1), -5), (dict(nb=0), -5), (dict(kc=8), -1),
    (dict(qo=None), -1), (dict(acc=None), -1), (dict(bt=None), -1), (dict(out=16), -1),
    (dict(out=None), -1), (dict(kf=16), -1), (dict(kf=16, vf=16, D=64), -3),
])
def test_compact_refuses(lib, kw, code):
    assert lib.paged_kv_compact(*dict(COMPACT, **kw).values()) == code


FORK = dict(kc=16, vc=16, kf=None, vf=None, bt=16, sl=16, par=16, kid=16, refs=16, free=16, count=4,
            left=4, refused=None, n=2, rows=4, H_kv=2, D=128, maxb=4, BS=16, cap=8, nb=9,
            stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(H_kv=0), -2), (dict(D=96), -3), (dict(BS=64), -4), (dict(n=-1), -5), (dict(rows=-1), -5),
    (dict(maxb=0), -5), (dict(cap=-1), -5), (dict(nb=0), -5), (dict(vc=None), -1),
    (dict(bt=None), -1), (dict(sl=8), -1), (dict(par=None), -1), (dict(kid=None), -1),
    (dict(refs=None), -1), (dict(free=None), -1), (dict(count=None), -1), (dict(left=2), -1),
    (dict(refused=2), -1), (dict(vf=16), -1),
])
def test_fork_refuses(lib, kw, code):
    assert lib.paged_kv_fork(*dict(FORK, **kw).values()) == code


RELEASE = dict(bt=16, sl=16, keep=16, refs=None, nb=0, free=16, count=4, out=16, left=4, n=2, maxb=4,
               BS=16, cap=8, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(BS=8), -4), (dict(n=-1), -5), (dict(maxb=0), -5), (dict(cap=-1), -5),
    (dict(n=2 ** 20, maxb=2 ** 12), -5), (dict(refs=16, nb=0), -5), (dict(refs=8, nb=4), -1),
    (dict(bt=None), -1), (dict(sl=None), -1), (dict(keep=8), -1), (dict(out=None), -1),
    (dict(free=None), -1), (dict(count=None), -1), (dict(left=6), -1),
])
def test_release_refuses(lib, kw, code):
    assert lib.paged_kv_release(*dict(RELEASE, **kw).values()) == code


def test_calls_without_rows_or_sequences_are_no_ops(lib):
    none = dict(q=None, k=None, v=None, out=None)
    for kw in (dict(total_q=0), dict(num_seqs=0)):
        a = dict(TREE, **none, qo=None, mask=None, bt=None, sl=None)
        a.update(kw)
        assert lib.paged_attn_decode_tree(*a.values()) == 0
    a = dict(ROPE, **none)
    a.update(rows=0)
    assert lib.paged_kv_rope_append_slots(*a.values()) == 0
    assert lib.paged_kv_compact(*dict(COMPACT, n=0, kc=None, out=None).values()) == 0


def test_the_status_has_a_text():
    assert "rotary_dim" in pa.paged_attn_status_string(-12)


def caches(dtype=BF):
    return torch.zeros(10, 2, 16, 128, dtype=dtype), torch.zeros(10, 2, 16, 128, dtype=dtype)


def tree():
    q = torch.zeros(3, 8, 128, dtype=BF)
    return [q, *caches(), torch.zeros(3, dtype=I32), torch.zeros(3, 1, dtype=I32),
            torch.zeros(2, 4, dtype=I32), torch.ones(2, dtype=I32), 0.1]


@pytest.mark.parametrize("at,bad", [
    (3, torch.zeros(2, dtype=I32)), (3, torch.zeros(3, dtype=torch.int64)),
    (4, torch.zeros(3, dtype=I32)), (4, torch.zeros(2, 1, dtype=I32)),
    (4, torch.zeros(3, 1, dtype=torch.int64)), (4, torch.zeros(1, 3, dtype=I32).t()[:, :0]),
    (0, torch.zeros(3, 8, 64, dtype=BF)), (5, torch.zeros(2, 4)), (6, torch.ones(2, 1, dtype=I32)),
])
def test_the_binding_refuses_other_trees(at, bad):
    a = tree()
    a[at] = bad
    with pytest.raises((ValueError, pa.PagedAttnError)):
        pa.paged_attn_decode_tree(*a)


def test_the_binding_refuses_unpinned_host_trees():
    with pytest.raises(ValueError, match="pinned"):
        pa.paged_attn_decode_tree(*tree())


def rope():
    q, kv = torch.zeros(3, 8, 128, dtype=BF), torch.zeros(3, 2, 128, dtype=BF)
    return dict(q=q, k_new=kv, v_new=kv.clone(), k_cache=caches()[0], v_cache=caches()[1],
                slot_map=torch.zeros(3, dtype=torch.int64), positions=torch.zeros(3, dtype=I32),
                cos_sin=torch.zeros(5, 64))


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(3, 8, 64, dtype=BF)), dict(q=torch.zeros(3, 8, 128)),
    dict(q=torch.zeros(3, 128, 8, dtype=BF).transpose(1, 2)),
    dict(k_new=torch.zeros(3, 4, 128, dtype=BF)), dict(v_new=torch.zeros(2, 2, 128, dtype=BF)),
    dict(k_new=torch.zeros(3, 4, 128, dtype=BF)[:, ::2]),
    dict(slot_map=torch.zeros(3, dtype=I32)), dict(positions=torch.zeros(4, dtype=I32)),
    dict(positions=torch.zeros(3, dtype=torch.int64)), dict(positions=torch.zeros(2, 4, dtype=I32)),
    dict(cos_sin=torch.zeros(64)), dict(cos_sin=torch.zeros(5, 64, dtype=torch.float64)),
    dict(freq_axis=torch.zeros(64, dtype=I32)), dict(freq_axis=torch.zeros(32)),
    dict(q_norm=torch.ones(64)), dict(k_norm=torch.ones(128, dtype=BF)),
    dict(k_scale=torch.zeros(10, 2, 16)), dict(out=torch.zeros(3, 8, 128)),
    dict(k_scale=torch.zeros(10, 2, 16), v_scale=torch.zeros(10, 2, 16)),
    dict(k_cache=torch.zeros(10, 2, 16, 128)),
])
def test_the_binding_refuses_other_rows_to_rotate(kw):
    with pytest.raises(ValueError) as e:
        pa.paged_kv_rope_append_slots(**dict(rope(), **kw))
    assert "pinned" not in str(e.value)


def pages():
    return dict(k_cache=caches()[0], v_cache=caches()[1], block_tables=torch.zeros(2, 4, dtype=I32),
                seq_lens=torch.ones(2, dtype=I32))


@pytest.mark.parametrize("kw", [
    dict(accepted=torch.zeros(2, dtype=I32)), dict(accepted=torch.zeros(3, 4, dtype=I32)),
    dict(accepted=torch.zeros(2, 4, dtype=torch.int64)), dict(qo_indptr=torch.zeros(2, dtype=I32)),
    dict(block_tables=torch.zeros(8, dtype=I32)), dict(seq_lens_out=torch.zeros(3, dtype=I32)),
    dict(k_scale=torch.zeros(10, 2, 16)), dict(v_cache=torch.zeros(10, 2, 16, 64, dtype=BF)),
])
def test_the_binding_refuses_other_compactions(kw):
    good = dict(pages(), qo_indptr=torch.zeros(3, dtype=I32), accepted=torch.zeros(2, 4, dtype=I32))
    with pytest.raises(ValueError) as e:
        pa.paged_kv_compact(**dict(good, **kw))
    assert "pinned" not in str(e.value)


@pytest.mark.parametrize("kw", [
    dict(children=torch.zeros(2, dtype=I32)), dict(parents=torch.zeros(1, dtype=torch.int64)),
    dict(block_refs=torch.zeros(9, dtype=I32)), dict(free_count=torch.zeros(2, dtype=I32)),
    dict(free_blocks=torch.zeros(4)), dict(refused=torch.zeros(1)),
    dict(seq_lens=torch.ones(3, dtype=I32)), dict(free_count_out=torch.zeros(1)),
    dict(k_cache=torch.zeros(10, 2, 16, 128, dtype=torch.uint8)),
])
def test_the_binding_refuses_other_forks(kw):
    one = torch.zeros(1, dtype=I32)
    good = dict(pages(), parents=one, children=one + 1, block_refs=torch.zeros(10, dtype=I32),
                free_blocks=torch.zeros(4, dtype=I32), free_count=one)
    with pytest.raises(ValueError) as e:
        pa.paged_kv_fork(**dict(good, **kw))
    assert "pinned" not in str(e.value)


@pytest.mark.parametrize("kw,name", [
    (dict(keep_lens=torch.zeros(3, dtype=I32)), "keep_lens"), (dict(block_size=2 ** 32 + 16), "block_size"),
    (dict(block_refs=torch.zeros(4)), "block_refs"), (dict(block_tables=torch.zeros(4, dtype=I32)), "block_tables"),
    (dict(free_blocks=torch.zeros(4, 2, dtype=I32)), "free_blocks"), (dict(seq_lens_out=torch.zeros(2)), "seq_lens_out"),
    (dict(free_count=torch.zeros(1, dtype=torch.int64)), "free_count"),
])
def test_the_binding_refuses_other_releases(kw, name):
    p = pages()
    good = dict(block_tables=p["block_tables"], seq_lens=p["seq_lens"],
                keep_lens=torch.zeros(2, dtype=I32), free_blocks=torch.zeros(4, dtype=I32),
                free_count=torch.zeros(1, dtype=I32), block_size=16)
    with pytest.raises(ValueError, match=name):
        pa.paged_kv_release(**dict(good, **kw))


@pytest.mark.parametrize("args", [(4, -1, 8, 2, 128, 8, 16), (4, 5, 8, 2, 128, 8, 8), (4, 5, 6, 4, 128, 8, 16),
                                  (-1, 5, 8, 2, 128, 8, 16)])
def test_the_workspace_query_rejects_bad_sizes(lib, args):
    assert lib.paged_attn_tree_workspace_bytes(*args) == 0
