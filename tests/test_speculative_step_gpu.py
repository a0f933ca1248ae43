"""Speculative and parallel decoding as an engine runs it: prompts, forked samples, drafted
trees verified, accepted rows moved together and the pages behind given back -- against an
engine that appends the accepted tokens alone, whose cache rows must be the same bits."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_decode_gb300 as pa
from oracle import serving, speculative as sp

pytestmark = pytest.mark.gpu

H_Q, H_KV, D, BS, MAXB, VOCAB, SCALE = 8, 2, 128, 16, 12, 97, float(np.float32(0.09))
DEV = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_decode_gb300 import build

    build.build()
    pa.load()


def i32(x):
    return torch.tensor(np.asarray(x), **DEV)


class Model:
    """One layer: a token's projections come from a table; norms and a rotation."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.qkv = torch.randn(VOCAB, (H_Q + 2 * H_KV) * D, generator=g, device="cuda").to(torch.bfloat16)
        angle = torch.arange(400, device="cuda", dtype=torch.float64)[:, None] * 500.0 ** (
            -torch.arange(D // 2, device="cuda", dtype=torch.float64) / (D // 2))
        self.cs = torch.cat([angle.cos(), angle.sin()], 1).float()
        self.qn, self.kn = (1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2))

    def rows(self, tokens):
        x = self.qkv[tokens]
        return (x[:, :H_Q * D].unflatten(1, (H_Q, D)), x[:, H_Q * D:(H_Q + H_KV) * D].unflatten(1, (H_KV, D)),
                x[:, (H_Q + H_KV) * D:].unflatten(1, (H_KV, D)))


class Engine:
    def __init__(self, rows, seed, nb=160, fp8=False):
        self.rows, self.nb = rows, nb
        if fp8:
            self.k, self.v = (torch.full((nb, H_KV, BS, D), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2))
            f = [torch.full((nb, H_KV, BS), float("nan"), device="cuda") for _ in range(2)]
            self.floats = dict(k_scale=f[0], v_scale=f[1])
        else:
            self.k, self.v = (torch.full((nb, H_KV, BS, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                              for _ in range(2))
            self.floats = {}
        self.table, self.lens = torch.zeros(rows, MAXB, **DEV), torch.zeros(rows, **DEV)
        self.refs = torch.zeros(nb, **DEV)
        self.free = i32(np.random.default_rng(seed).permutation(nb))
        self.count = i32([nb])

    def append(self, m, new, tokens, positions, **kw):
        """Blocks, rotated rows in the cache and queries of new tokens (list of counts)."""
        total = int(sum(new))
        _, qo, slots, _ = pa.paged_kv_assign(self.lens, i32(new), self.table, self.free, self.count, BS, total,
                                             seq_lens_out=self.lens, free_count_out=self.count)
        q, k, v = m.rows(torch.as_tensor(tokens, device="cuda"))
        q = pa.paged_kv_rope_append_slots(q, k, v, self.k, self.v, slots, i32(positions), m.cs, q_norm=m.qn,
                                          k_norm=m.kn, **self.floats, **kw)
        return q, qo

    def content(self):
        """Rows of each sequence, as bits."""
        lens, table = self.lens.cpu().numpy(), self.table.cpu().numpy()
        out = []
        for c in (self.k, self.v, *self.floats.values()):
            c = c.cpu()
            c = c.view(torch.int16).numpy() if c.dtype is torch.bfloat16 else c.numpy()
            c = c[..., None] if c.ndim == 3 else c
            out.append([serving.rows_of(c, table[s], lens[s]) for s in range(self.rows)])
        return out

    def check_blocks(self):
        """Each block is held as often as it is counted, or is on the stack once."""
        lens, table, refs = (x.cpu().numpy() for x in (self.lens, self.table, self.refs))
        held = np.bincount(np.concatenate([table[s, :-(-lens[s] // BS)] for s in range(self.rows)]).astype(np.int64),
                           minlength=self.nb)
        free = np.bincount(self.free.cpu().numpy()[:int(self.count)].astype(np.int64), minlength=self.nb)
        assert (refs == np.maximum(held - 1, 0)).all() and (free == (held == 0)).all()


def draft(rng, widest):
    """A tree: parents, its mask bits, depths."""
    m = int(rng.integers(1, widest + 1))
    parent = [int(rng.integers(-1, j)) if j else -1 for j in range(m)]
    bits = np.zeros((m, m), dtype=bool)
    for j, p in enumerate(parent):
        if p >= 0:
            bits[j] = bits[p]
        bits[j, j] = True
    return bits, bits.sum(1) - 1


def accept(rng, bits):
    """The path to a random node, or nothing."""
    j = int(rng.integers(-1, len(bits)))
    return np.nonzero(bits[j])[0] if j >= 0 else np.zeros(0, dtype=int)


@pytest.mark.parametrize("fp8", [False, True])
def test_trees_leave_what_plain_decoding_leaves(fp8):
    rng, m = np.random.default_rng(3), Model(4)
    rows, prompts = 9, [40, 1, 33]
    a, b = Engine(rows, 5, fp8=fp8), Engine(rows, 6, fp8=fp8)
    tokens = rng.integers(0, VOCAB, size=sum(prompts))
    new = prompts + [0] * (rows - len(prompts))
    where = np.concatenate([np.arange(n) for n in prompts])
    for e in (a, b):
        e.append(m, new, tokens, where)
        # two samples more of each prompt
        pa.paged_kv_fork(e.k, e.v, e.table, e.lens, i32([0, 0, 1, 1, 2, 2]), i32([3, 4, 5, 6, 7, 8]), e.refs, e.free,
                         e.count, free_count_out=e.count, **e.floats)
        e.check_blocks()
    for step in range(6):
        trees = [draft(rng, 40) for _ in range(rows)]
        ql = [len(t[0]) for t in trees]
        drafted = [rng.integers(0, VOCAB, size=n) for n in ql]
        ctx = a.lens.cpu().numpy()
        q, qo = a.append(m, ql, np.concatenate(drafted), np.concatenate([ctx[s] + t[1] for s, t in enumerate(trees)]))
        mask = np.concatenate([sp.mask_words(t[0], 2) for t in trees])
        if not fp8:
            out = pa.paged_attn_decode_tree(q, a.k, a.v, qo, i32(mask), a.table, a.lens, SCALE, softcap=30.0)
            res = sp.attend_tree(serving.bf16_to_f64(q), serving.bf16_to_f64(a.k), serving.bf16_to_f64(a.v),
                                 qo.cpu().numpy(), mask, a.table.cpu().numpy(), a.lens.cpu().numpy(), SCALE,
                                 softcap=30.0)
            assert (np.abs(serving.bf16_to_f64(out) - res.out) <= res.tol).all()
        paths = [accept(rng, t[0]) for t in trees]
        lists = np.full((rows, 41), -1, dtype=np.int64)
        for s, p in enumerate(paths):
            lists[s, :len(p)] = p
        kept = pa.paged_kv_compact(a.k, a.v, qo, i32(lists), a.table, a.lens, **a.floats)
        pa.paged_kv_release(a.table, a.lens, kept, a.free, a.count, BS, block_refs=a.refs, seq_lens_out=a.lens,
                            free_count_out=a.count)
        # the other engine appends the accepted tokens alone
        n = [len(p) for p in paths]
        if sum(n):
            b.append(m, n, np.concatenate([d[p] for d, p in zip(drafted, paths)]),
                     np.concatenate([ctx[s] + np.arange(len(p)) for s, p in enumerate(paths)]))
        torch.cuda.synchronize()
        assert torch.equal(a.lens, b.lens)
        for x, y in zip(a.content(), b.content()):
            for s in range(rows):
                assert np.array_equal(x[s].view(np.int32) if x[s].dtype == np.float32 else x[s],
                                      y[s].view(np.int32) if y[s].dtype == np.float32 else y[s])
        a.check_blocks()
        b.check_blocks()
        if step == 3:  # half of the samples end, and one starts again from another
            for e in (a, b):
                keep = e.lens.clone()
                keep[1::2] = 0
                pa.paged_kv_release(e.table, e.lens, keep, e.free, e.count, BS, block_refs=e.refs, seq_lens_out=e.lens,
                                    free_count_out=e.count)
                pa.paged_kv_fork(e.k, e.v, e.table, e.lens, i32([2, 2]), i32([5, 1]), e.refs, e.free, e.count,
                                 free_count_out=e.count, **e.floats)
                e.check_blocks()
    one = torch.randn(rows, H_Q, D, device="cuda").to(torch.bfloat16)
    if fp8:
        outs = [pa.paged_attn_decode_fp8(one, e.k, e.v, e.floats["k_scale"], e.floats["v_scale"], e.table, e.lens, SCALE)
                for e in (a, b)]
    else:
        outs = [pa.paged_attn_decode(one, e.k, e.v, e.table, e.lens, SCALE) for e in (a, b)]
    assert torch.equal(*outs)


def test_a_captured_step_replays_with_new_trees():
    """Assign, rotate and append, attend, compact, release in one graph, on a stream of its own."""
    rng, m = np.random.default_rng(7), Model(8)
    rows, each = 4, 12
    total = rows * each
    a, b = Engine(rows, 9), Engine(rows, 9)
    prompt = rng.integers(0, VOCAB, size=4 * 20)
    for e in (a, b):
        e.append(m, [20] * rows, prompt, np.tile(np.arange(20), rows))
    new = i32([each] * rows)
    pos, mask, acc = torch.zeros(total, **DEV), torch.zeros(total, 1, **DEV), torch.zeros(rows, each, **DEV)
    x = torch.zeros(total, m.qkv.shape[1], dtype=torch.bfloat16, device="cuda")
    q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([H_Q * D, H_KV * D, H_KV * D], dim=1))
    qo, slots = torch.zeros(rows + 1, **DEV), torch.zeros(total, dtype=torch.int64, device="cuda")
    rot, out, kept = (torch.empty(total, H_Q, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)), None, torch.zeros(rows, **DEV)
    rot, out = rot
    ws = torch.zeros(pa.paged_attn_tree_workspace_bytes(rows, total, H_Q, H_KV, D, MAXB, BS), dtype=torch.uint8, device="cuda")

    def step(e):
        pa.paged_kv_assign(e.lens, new, e.table, e.free, e.count, BS, total, seq_lens_out=e.lens, qo_indptr=qo,
                           slot_map=slots, free_count_out=e.count)
        pa.paged_kv_rope_append_slots(q, k, v, e.k, e.v, slots, pos, m.cs, q_norm=m.qn, k_norm=m.kn, out=rot)
        pa.paged_attn_decode_tree(rot, e.k, e.v, qo, mask, e.table, e.lens, SCALE, out=out, workspace=ws)
        pa.paged_kv_compact(e.k, e.v, qo, acc, e.table, e.lens, seq_lens_out=kept)
        pa.paged_kv_release(e.table, e.lens, kept, e.free, e.count, BS, block_refs=e.refs, seq_lens_out=e.lens,
                            free_count_out=e.count)

    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        step(a)
    for _ in range(5):
        ctx = a.lens.cpu().numpy()
        bits = [draft(rng, each)[0] for _ in range(rows)]
        full = np.zeros((total, each), dtype=bool)  # shorter trees: padding nodes behind
        depth, lists = np.zeros(total, dtype=int), np.full((rows, each), -1)
        for s, t in enumerate(bits):
            full[s * each:s * each + len(t), :len(t)] = t
            depth[s * each:(s + 1) * each] = ctx[s]
            depth[s * each:s * each + len(t)] += t.sum(1) - 1
            p = accept(rng, t)
            lists[s, :len(p)] = p
        mask.copy_(i32(sp.mask_words(full, 1)))
        pos.copy_(i32(depth))
        acc.copy_(i32(lists))
        x.copy_(m.qkv[torch.as_tensor(rng.integers(0, VOCAB, size=total), device="cuda")])
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step(b)
        torch.cuda.synchronize()
        assert torch.equal(got, out) and torch.equal(a.lens, b.lens)
        for u, w in zip(a.content(), b.content()):
            assert all(np.array_equal(i, j) for i, j in zip(u, w))
        a.check_blocks()


def test_calls_on_two_streams_at_once():
    """Each stream has its own engine; nothing is shared but the library's workspaces."""
    rng, m = np.random.default_rng(11), Model(12)
    alone, together = [], []
    for pair in (alone, together):
        for i in range(2):
            e = Engine(6, 13 + i)
            e.append(m, [60] * 6, np.arange(360) * (i + 3) % VOCAB, np.tile(np.arange(60), 6))
            pair.append(e)
    bits = [draft(rng, 20)[0] for _ in range(6)]
    mask = i32(np.concatenate([sp.mask_words(t, 1) for t in bits]))
    ql = [len(t) for t in bits]
    qo = i32(np.concatenate([[0], np.cumsum(ql)]))
    q = torch.randn(sum(ql), H_Q, D, device="cuda").to(torch.bfloat16)
    lists = np.full((6, 20), -1)
    for s, t in enumerate(bits):
        p = accept(rng, t)
        lists[s, :len(p)] = p
    lists = i32(lists)
    torch.cuda.synchronize()

    def work(e):
        outs = []
        for _ in range(5):
            outs.append(pa.paged_attn_decode_tree(q, e.k, e.v, qo, mask, e.table, e.lens, SCALE))
            kept = pa.paged_kv_compact(e.k, e.v, qo, lists, e.table, e.lens)
            pa.paged_kv_release(e.table, e.lens, kept, e.free, e.count, BS, block_refs=e.refs, free_count_out=e.count.clone())
        return outs

    want = [work(e) for e in alone]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for e, st in zip(together, streams):
        with torch.cuda.stream(st):
            got.append(work(e))
    torch.cuda.synchronize()
    for w, x in zip(want, got):
        assert all(torch.equal(i, j) for i, j in zip(w, x))
    for e, f in zip(alone, together):
        assert torch.equal(e.k.view(torch.int16), f.k.view(torch.int16)) and torch.equal(e.free, f.free)
