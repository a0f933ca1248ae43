"""The serving operators as an engine runs them: blocks assigned, rows appended by slot,
attention over what the cache then holds -- prompts, then decode steps, also captured,
on a stream of their own, and two at once."""
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


H_Q, H_KV, D, BS, MAXB = 8, 2, 128, 16, 12
SCALE = float(np.float32(0.09))


class Engine:
    """A cache and its bookkeeping on the GPU, and the same on the host in float64."""

    def __init__(self, n, seed, nb=120):
        self.n, self.nb = n, nb
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        dev = dict(dtype=torch.int32, device="cuda")
        self.k = torch.full((nb, H_KV, BS, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        self.lens, self.count = torch.zeros(n, **dev), torch.tensor([nb], **dev)
        self.table = torch.zeros(n, MAXB, **dev)
        self.h_free = self.rng.permutation(nb)
        self.free = torch.tensor(self.h_free, **dev)
        self.h_lens, self.h_count = np.zeros(n, dtype=np.int64), nb
        self.h_table = np.zeros((n, MAXB), dtype=np.int64)
        self.h_k = np.full((nb, H_KV, BS, D), np.nan)
        self.h_v = self.h_k.copy()

    def rows(self, total):
        """A fused projection's output, as (q, k, v)."""
        x = torch.randn(total, (H_Q + 2 * H_KV) * D, generator=self.g, device="cuda").to(torch.bfloat16)
        q, k, v = x.split([H_Q * D, H_KV * D, H_KV * D], dim=1)
        return (q.unflatten(1, (H_Q, D)).contiguous(), k.unflatten(1, (H_KV, D)),
                v.unflatten(1, (H_KV, D)))

    def host(self, new, q, k, v):
        total = int(sum(new))
        self.h_lens, qo, slots, self.h_count, refused, self.h_table = serving.assign(
            self.h_lens, new, self.h_table, self.h_free, self.h_count, BS, total)
        assert refused == 0
        for r, s in enumerate(slots):
            self.h_k[s // BS, :, s % BS] = serving.bf16_to_f64(k[r])
            self.h_v[s // BS, :, s % BS] = serving.bf16_to_f64(v[r])
        return qo

    def check(self, out, q, qo, **kw):
        res = serving.attend(serving.bf16_to_f64(q), self.h_k, self.h_v, qo, self.h_table,
                             self.h_lens, SCALE, **kw)
        err = np.abs(serving.bf16_to_f64(out) - res.out)
        assert (err <= res.tol).all(), (err / np.maximum(res.tol, 1e-300)).max()


def step(e, d_new, total, q, k, v, stream=None, qo=None, slots=None, out=None, ws=None, **kw):
    _, qo, slots, _ = pa.paged_kv_assign(
        e.lens, d_new, e.table, e.free, e.count, BS, total, seq_lens_out=e.lens, qo_indptr=qo,
        slot_map=slots, free_count_out=e.count, stream=stream)
    pa.paged_kv_append_slots(k, v, e.k, e.v, slots, stream=stream)
    return pa.paged_attn_decode_multi_mods(q, e.k, e.v, qo, e.table, e.lens, SCALE, out=out,
                                           workspace=ws, stream=stream, **kw)


OPTS = dict(softcap=20.0, window=100)


@pytest.mark.parametrize("n,seed", [(1, 1), (5, 2), (9, 3)])
def test_prompts_then_decode_steps(n, seed):
    e = Engine(n, seed)
    new = np.array([int(x) for x in e.rng.integers(1, 90, size=n)])
    for t in range(6):
        total = int(new.sum())
        q, k, v = e.rows(total)
        out = step(e, torch.tensor(new, dtype=torch.int32, device="cuda"), total, q, k, v, **OPTS)
        torch.cuda.synchronize()
        qo = e.host(new, q, k, v)
        e.check(out, q, qo, **OPTS)
        if (new == 1).all():  # the single-token entry point gives the same step
            one = pa.paged_attn_decode_mods(q, e.k, e.v, e.table, e.lens, SCALE, **OPTS)
            e.check(one, q, qo, **OPTS)
        new = np.ones(n, dtype=int) if t != 2 else np.array([int(x) for x in e.rng.integers(0, 7, size=n)])


def test_a_captured_decode_step_replayed():
    e = Engine(4, 7)
    q, k, v = e.rows(150)
    first = np.array([70, 15, 16, 49])
    step(e, torch.tensor(first, dtype=torch.int32, device="cuda"), 150, q, k, v)
    e.host(first, q, k, v)
    ones = torch.ones(4, dtype=torch.int32, device="cuda")
    q, k, v = e.rows(4)
    x = torch.cat([k, v], dim=1).contiguous()     # static buffers of the captured step
    kb, vb = x[:, :H_KV], x[:, H_KV:]
    out = torch.zeros_like(q)
    qo = torch.zeros(5, dtype=torch.int32, device="cuda")
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    ws = torch.zeros(pa.paged_attn_multi_mods_workspace_bytes(4, 4, H_Q, H_KV, D, MAXB, BS),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(e, ones, 4, q, kb, vb, qo=qo, slots=slots, out=out, ws=ws, **OPTS)
    for _ in range(5):
        nq, nk, nv = e.rows(4)
        q.copy_(nq)
        kb.copy_(nk)
        vb.copy_(nv)
        graph.replay()
        torch.cuda.synchronize()
        e.check(out, q, e.host([1] * 4, nq, nk, nv), **OPTS)


def test_two_streams_at_once_with_their_own_workspaces():
    engines = [Engine(3, 11), Engine(5, 12)]
    streams = [torch.cuda.Stream() for _ in engines]
    new = [np.array([40, 100, 7]), np.array([1, 90, 33, 64, 16])]
    rows = [e.rows(int(m.sum())) for e, m in zip(engines, new)]
    d_new = [torch.tensor(m, dtype=torch.int32, device="cuda") for m in new]
    ws = [torch.zeros(pa.paged_attn_multi_mods_workspace_bytes(e.n, int(m.sum()), H_Q, H_KV, D,
                                                               MAXB, BS),
                      dtype=torch.uint8, device="cuda") for e, m in zip(engines, new)]
    torch.cuda.synchronize()
    outs = []
    for e, s, m, r, d, w in zip(engines, streams, new, rows, d_new, ws):
        with torch.cuda.stream(s):
            outs.append(step(e, d, int(m.sum()), *r, stream=s, ws=w, **OPTS))
    torch.cuda.synchronize()
    for e, m, r, o in zip(engines, new, rows, outs):
        e.check(o, r[0], e.host(m, *r), **OPTS)


def test_chats_over_a_prompt_that_was_written_by_the_same_operators():
    """One prompt's blocks become the shared prefix of three chats."""
    e = Engine(4, 13)
    prompt = np.array([83, 0, 0, 0])
    q, k, v = e.rows(83)
    step(e, torch.tensor(prompt, dtype=torch.int32, device="cuda"), 83, q, k, v)
    e.host(prompt, q, k, v)
    chats = np.array([0, 20, 1, 37])
    q, k, v = e.rows(58)
    step(e, torch.tensor(chats, dtype=torch.int32, device="cuda"), 58, q, k, v)
    e.host(chats, q, k, v)
    last = torch.randn(3, H_Q, D, generator=e.g, device="cuda").to(torch.bfloat16)
    out = pa.paged_attn_decode_shared(
        last, e.k, e.v, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), e.table[:1],
        e.lens[:1], e.table[1:].clone(), e.lens[1:].clone(), SCALE, softcap=20.0)
    torch.cuda.synchronize()
    res = serving.attend_shared(serving.bf16_to_f64(last), e.h_k, e.h_v, [0, 3], e.h_table[:1],
                                e.h_lens[:1], e.h_table[1:], e.h_lens[1:], SCALE, 20.0)
    err = np.abs(serving.bf16_to_f64(out) - res.out)
    assert (err <= res.tol).all()


def test_offsets_that_fall_are_reported_and_nothing_is_read_or_written_outside():
    e = Engine(3, 14)
    new = np.array([20, 30, 10])
    q, k, v = e.rows(60)
    step(e, torch.tensor(new, dtype=torch.int32, device="cuda"), 60, q, k, v)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    guard = torch.full((62, H_Q, D), 5.0, dtype=torch.bfloat16, device="cuda")
    try:
        pa.paged_attn_set_checks(e.nb, status)
        for qo, bits in (([0, 20, 50, 60], 0), ([0, 30, 20, 60], 2), ([0, 20, 50, 90], 2),
                         ([-4, 20, 50, 60], 2)):
            status.zero_()
            pa.paged_attn_decode_multi_mods(q, e.k, e.v, torch.tensor(qo, dtype=torch.int32).cuda(),
                                            e.table, e.lens, SCALE, out=guard[1:61])
            torch.cuda.synchronize()
            assert int(status) == bits, qo
            assert (guard[0] == 5.0).all() and (guard[61] == 5.0).all()
    finally:
        pa.paged_attn_set_checks(0, None)
