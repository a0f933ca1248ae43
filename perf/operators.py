"""Cases of the serving operators around the paged KV cache, with their plain forms.

Five operators of one serving step, as an engine calls them in order:

* ``assign``  -- block tables, the ragged query offsets and the slot map of the
  new tokens, built on the GPU from request lengths and a free list;
* ``append``  -- the new tokens' K and V rows written to the cache by slot;
* ``decode``  -- one query token per sequence over a bf16 or FP8 cache, with
  capped scores, a distance bias, a window, a prefix and documents;
* ``multi``   -- the same for several query tokens per sequence (verification of
  drafted tokens, chunks of a prompt);
* ``shared``  -- one query token per sequence of groups that share a long prefix.

``run`` computes an operator in elementary torch operations in 32 bits, or, when
``own`` is true, through the framework's entry points.  A query at position
``pos`` sees token t of its L tokens when t < prefix, or when t is at or after
both the start of the query's document and pos - window + 1 and (causally) not
after pos.  Its score is cap * tanh(scale * q.k / cap) - slope[head] * |pos - t|.
"""
import math

import numpy as np
import torch

own = False

# softcap 0, window 0, alibi False, prefix 0, doc 0: that part is off
_ATTN = dict(softcap=0.0, window=0, alibi=False, prefix=0, doc=0, causal=True)


def listed():
    llama = dict(heads=32, kv_heads=8, dim=128, page=16)
    wide = dict(heads=24, kv_heads=4, dim=256, page=16)
    return [
        # two short chats in a capped, windowed layer: a call whose latency counts
        dict(_ATTN, name="decode_tiny", op="decode", fp8=False, seqs=2, len_lo=37, len_hi=100,
             heads=4, kv_heads=2, dim=64, page=16, softcap=30.0, window=64),
        # a decode step of a windowed layer with capped scores and four sink tokens
        dict(_ATTN, **llama, name="decode_window", op="decode", fp8=False, seqs=32, len_lo=512,
             len_hi=4096, softcap=50.0, window=1024, prefix=4),
        # a large ragged batch over an FP8 cache with a distance bias and packed documents
        dict(_ATTN, **llama, name="decode_fp8_ragged", op="decode", fp8=True, seqs=128, len_lo=16,
             len_hi=8192, alibi=True, doc=6000),
        # verification of five drafted tokens per sequence, capped scores
        dict(_ATTN, **llama, name="multi_verify", op="multi", seqs=32, len_lo=512, len_hi=4096,
             q_lo=5, q_hi=5, softcap=50.0),
        # prompt chunks of four requests in a windowed, capped layer
        dict(_ATTN, **llama, name="multi_chunk", op="multi", seqs=4, len_lo=5003, len_hi=8192,
             q_lo=1500, q_hi=2048, softcap=50.0, window=4096),
        # chunks of two long packed prompts with a bidirectional prefix and a distance bias
        dict(_ATTN, **wide, name="multi_prefix_d256", op="multi", seqs=2, len_lo=15001, len_hi=20000,
             q_lo=300, q_hi=512, alibi=True, prefix=2000, doc=9000),
        # three system prompts under 64 chats
        dict(**llama, name="shared_prompts", op="shared", seqs=64, groups=3, pre_lo=2001, pre_hi=8192,
             len_lo=1, len_hi=1024, softcap=0.0, alibi=False),
        # sixteen questions to one document of 100000 tokens
        dict(**wide, name="shared_document", op="shared", seqs=16, groups=1, pre_lo=100000,
             pre_hi=100000, len_lo=64, len_hi=2000, softcap=0.0, alibi=False),
        # the bookkeeping of a decode step: one new token for each of 256 requests
        dict(name="assign_step", op="assign", seqs=256, page=16, len_lo=16, len_hi=32768, new_lo=1,
             new_hi=1),
        # admission of 512 prompts
        dict(name="assign_prompts", op="assign", seqs=512, page=16, len_lo=0, len_hi=0, new_lo=16,
             new_hi=8192),
        # the new rows of a decode step, slices of one fused projection
        dict(name="append_step", op="append", rows=256, kv_heads=8, heads=32, dim=128, page=16,
             blocks=8192),
        # the rows of a prefill step
        dict(name="append_prompts", op="append", rows=8192, kv_heads=8, heads=32, dim=128, page=16,
             blocks=16384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "multi", "multi", "shared", "assign", "append"])
    if op == "assign":
        seqs = _log(rng, 1, 2048)
        new_hi = _log(rng, 1, max(1, 1000000 // seqs))
        new_hi = min(new_hi, 8192)
        return dict(op=op, seqs=seqs, page=rng.choice([16, 32]), len_lo=0,
                    len_hi=_log(rng, 16, 32768), new_lo=rng.randint(0, new_hi), new_hi=new_hi)
    kv_heads = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128, 256])
    shape = dict(kv_heads=kv_heads, heads=kv_heads * rng.choice([1, 2, 4, 5, 6, 8, 16]), dim=dim,
                 page=rng.choice([16, 32]))
    if op == "append":
        return dict(shape, op=op, rows=_log(rng, 1, 8192 if dim < 256 else 4096),
                    blocks=_log(rng, 1024, 8192))
    shape["softcap"] = rng.choice([0.0, 30.0, 50.0])
    shape["alibi"] = rng.random() < 0.4
    if op == "shared":
        seqs = _log(rng, 1, 64)
        pre = _log(rng, 16, 100000 if dim * kv_heads <= 512 else 16384)
        return dict(shape, op=op, seqs=seqs, groups=rng.randint(1, min(seqs, 4)),
                    pre_lo=max(1, pre // rng.randint(1, 4)), pre_hi=pre, len_lo=rng.randint(0, 5),
                    len_hi=_log(rng, 16, 1024))
    shape.update(window=rng.choice([0, 0, _log(rng, 16, 4096)]),
                 prefix=rng.choice([0, 0, 4, _log(rng, 1, 2048)]),
                 doc=rng.choice([0, 0, _log(rng, 100, 20000)]))
    if op == "decode":
        fp8 = dim >= 128 and rng.random() < 0.4
        seqs = _log(rng, 1, 128)
        len_hi = min(32768, _log(rng, 16, max(17, 1000000 * 128 * 8 // (seqs * kv_heads * dim))))
        return dict(shape, op=op, fp8=fp8, seqs=seqs, causal=True,
                    len_lo=rng.randint(1, min(100, len_hi)), len_hi=len_hi)
    seqs = _log(rng, 1, 32)
    len_hi = _log(rng, 16, 16384)
    room = 8e10 / (shape["heads"] * len_hi * seqs * dim)
    q_hi = max(1, min(len_hi, _log(rng, 1, 2048), int(room)))
    return dict(shape, op=op, seqs=seqs, len_lo=rng.randint(1, len_hi), len_hi=len_hi,
                q_lo=rng.randint(1, q_hi), q_hi=q_hi, causal=rng.random() < 0.8)


# ------------------------------------------------------------------ sizes of a case

def _spread(lo, hi, n, seed):
    """n lengths from hi down to lo, log-uniform between them; the same for every seed of a case."""
    rng = np.random.default_rng(seed)
    a = max(lo, 1)
    x = np.round(np.exp(rng.uniform(math.log(a), math.log(max(hi, a)), size=n))).astype(np.int64)
    x = np.clip(x, lo, hi)
    x[0] = hi
    if n > 1:
        x[-1] = lo
    return x


def _lens(case):
    return _spread(case["len_lo"], case["len_hi"], case["seqs"], 1)


def _q_lens(case):
    if case["op"] != "multi":
        return np.ones(case["seqs"], dtype=np.int64)
    return np.minimum(_spread(case["q_lo"], case["q_hi"], case["seqs"], 2), _lens(case))


def _prefixes(case):
    """Visible prefix of each sequence (decode, multi): not all the same."""
    lens = _lens(case)
    return np.minimum(lens, case["prefix"] + np.arange(len(lens)) % 5)


def _rows(case):
    """(sequence, position, first and last token inside the window and document) of each query."""
    lens, ql = _lens(case), _q_lens(case)
    seq = np.repeat(np.arange(len(lens)), ql)
    at = np.arange(len(seq)) - np.repeat(np.cumsum(ql) - ql, ql)
    pos = lens[seq] - ql[seq] + at
    lo = np.zeros_like(pos)
    if case["window"]:
        lo = np.maximum(lo, pos - case["window"] + 1)
    if case["doc"]:
        lo = np.maximum(lo, pos // case["doc"] * case["doc"])
    hi = pos if case["causal"] else lens[seq] - 1
    return seq, pos, lo, hi


def _group_sizes(case):
    n, g = case["seqs"], case["groups"]
    return np.array([n // g + (1 if i < n % g else 0) for i in range(g)], dtype=np.int64)


def _new_lens(case):
    return _spread(case["new_lo"], case["new_hi"], case["seqs"], 3)


def work(case):
    op = case["op"]
    if op == "assign":
        lens, new = _lens(case), _new_lens(case)
        pages = int((-(-(lens + new) // case["page"]) - -(-lens // case["page"])).sum())
        n = len(lens)
        # lengths in, lengths and offsets out, one slot per token, one id in and out per page
        return {"bytes": float(n * 8 + n * 4 + (n + 1) * 4 + int(new.sum()) * 8 + pages * 8 + 8),
                "flops": 0.0}
    D, H, K = case["dim"], case["heads"], case["kv_heads"]
    if op == "append":
        return {"bytes": float(case["rows"] * (8 + 2 * 2 * 2 * K * D)), "flops": 0.0}
    lens = _lens(case)
    if op == "shared":
        pre, size = _spread(case["pre_lo"], case["pre_hi"], case["groups"], 4), _group_sizes(case)
        tokens = int(pre.sum() + lens.sum())
        pairs = int((pre * size).sum() + lens.sum())
        rows = case["seqs"]
        row_bytes = 4 * D
    else:
        seq, pos, lo, hi = _rows(case)
        pre = _prefixes(case) if case["prefix"] else np.zeros_like(lens)
        seen = np.maximum(hi - lo + 1, 0) + np.minimum(pre[seq], lo) + np.maximum(pre[seq] - 1 - hi, 0)
        pairs = int(seen.sum())
        first = np.full(len(lens), 1 << 40)
        np.minimum.at(first, seq, lo)
        tokens = int((lens - first + np.minimum(pre, first)).sum())
        rows = len(seq)
        row_bytes = 2 * (D + 4) if case.get("fp8") else 4 * D
    return {"bytes": float(tokens * K * row_bytes + rows * H * D * 4 + (tokens // case["page"]) * 4),
            "flops": float(4 * D * H * pairs)}


# ------------------------------------------------------------------ inputs

def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _tables(rng, pages, first_block, maxb):
    """Block tables [n, maxb] with shuffled blocks; entries a sequence does not use hold a spare one."""
    total = int(pages.sum())
    ids = rng.permutation(total) + first_block
    bt = np.full((len(pages), maxb), first_block + total, dtype=np.int64)
    inside = np.arange(maxb)[None, :] < pages[:, None]
    bt[inside] = ids
    return bt


def _normal(shape, gen, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _to_fp8(x):
    """e4m3 bytes and one float per row."""
    f = x.float().abs().amax(-1) / 448.0
    f = torch.where(f > 0, f, torch.ones_like(f))
    return (x.float() / f[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), f


def _slopes(heads):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)],
                        dtype=torch.float32, device="cuda")


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, page = case["op"], case["page"]
    s = {"op": op, "page": page}
    if op == "assign":
        lens, new = _lens(case), _new_lens(case)
        old_pages = -(-lens // page)
        need = int((-(-(lens + new) // page) - old_pages).sum())
        free = need + 100
        maxb = int((-(-(lens + new) // page)).max()) + 3
        used = int(old_pages.sum())
        bt = _tables(rng, old_pages, 0, maxb)
        s.update(block_tables=_i32(bt), seq_lens=_i32(lens), new_lens=_i32(new),
                 free_blocks=_i32(rng.permutation(free) + used + 1), free_count=_i32([free]),
                 max_new=int(new.sum()) + 64)
        return s
    D, H, K = case["dim"], case["heads"], case["kv_heads"]
    if op == "append":
        rows, blocks = case["rows"], case["blocks"]
        qkv = _normal((rows, (H + 2 * K) * D), gen)  # a fused projection's output
        slots = rng.permutation(blocks * page)[:rows]
        slots[rng.random(rows) < 0.02] = -1           # padding rows of the step
        s.update(k_new=qkv[:, H * D:(H + K) * D].unflatten(1, (K, D)),
                 v_new=qkv[:, (H + K) * D:].unflatten(1, (K, D)),
                 slots=torch.tensor(slots, dtype=torch.int64, device="cuda"),
                 k_cache=_normal((blocks, K, page, D), gen),
                 v_cache=_normal((blocks, K, page, D), gen))
        return s
    lens = _lens(case)
    pages = -(-lens // page)
    maxb = max(1, int(pages.max()))
    s.update(scale=1.0 / math.sqrt(D), softcap=float(case["softcap"]),
             slopes=_slopes(H) if case["alibi"] else None, seq_lens=_i32(lens), heads=H, kv_heads=K)
    if op == "shared":
        pre = _spread(case["pre_lo"], case["pre_hi"], case["groups"], 4)
        pp = -(-pre // page)
        both = np.concatenate([pages, pp])
        wide = max(maxb, int(pp.max()))
        bt = _tables(rng, both, 0, wide)
        size = _group_sizes(case)
        blocks = int(both.sum()) + 1
        s.update(block_tables=_i32(np.ascontiguousarray(bt[:len(lens), :maxb])),
                 prefix_tables=_i32(bt[len(lens):]), prefix_lens=_i32(pre),
                 group_indptr=_i32(np.concatenate([[0], np.cumsum(size)])),
                 group=torch.tensor(np.repeat(np.arange(len(size)), size), device="cuda"),
                 member=torch.tensor(np.concatenate([np.arange(n) for n in size]), device="cuda"),
                 widest=int(size.max()), most=int(lens.max()), most_prefix=int(pre.max()))
        rows = case["seqs"]
    else:
        seq, pos, lo, hi = _rows(case)
        ql = _q_lens(case)
        blocks = int(pages.sum()) + 1
        s.update(block_tables=_i32(_tables(rng, pages, 0, maxb)), window=case["window"],
                 prefix_lens=_i32(_prefixes(case)) if case["prefix"] else None,
                 doc_starts=_i32(pos // case["doc"] * case["doc"]) if case["doc"] else None,
                 qo_indptr=_i32(np.concatenate([[0], np.cumsum(ql)])), causal=case["causal"],
                 seq=torch.tensor(seq, device="cuda"),
                 at=torch.tensor(pos - lens[seq] + ql[seq], device="cuda"), widest=int(ql.max()),
                 most=int(lens.max()))
        rows = len(seq)
    s["q"] = _normal((rows, H, D), gen)
    k, v = _normal((blocks, K, page, D), gen), _normal((blocks, K, page, D), gen)
    if case.get("fp8"):
        s["k_cache"], s["k_scale"] = _to_fp8(k)
        s["v_cache"], s["v_scale"] = _to_fp8(v)
    else:
        s["k_cache"], s["v_cache"] = k, v
    return s


# ------------------------------------------------------------------ the plain forms

def _plain_assign(s):
    """Blocks are taken from the top of the free stack, sequence by sequence; a sequence whose pages
    are not all there, or do not fit its table row, gets none, keeps its length and slots of -1."""
    page, bt = s["page"], s["block_tables"]
    old, new = s["seq_lens"].long(), s["new_lens"].long()
    n, maxb = bt.shape
    fits = old + new <= maxb * page
    old_pages = (old + page - 1) // page
    need = torch.where(fits, (old + new + page - 1) // page - old_pages, 0)
    end = need.cumsum(0)
    free = s["free_count"].long()
    given = fits & ((need == 0) | (end <= free))
    indptr = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
    indptr[1:] = new.cumsum(0)
    column = torch.arange(maxb, device="cuda")[None, :]
    fresh = given[:, None] & (column >= old_pages[:, None]) & (column < (old_pages + need)[:, None])
    place = free - 1 - ((end - need)[:, None] + column - old_pages[:, None])
    taken = s["free_blocks"][place.clamp(0, s["free_blocks"].numel() - 1)]
    bt.copy_(torch.where(fresh, taken, bt))
    row = torch.arange(s["max_new"], device="cuda")
    seq = torch.searchsorted(indptr[1:], row, right=True).clamp(max=n - 1)
    t = old[seq] + row - indptr[seq]
    block = bt[seq, (t // page).clamp(max=maxb - 1)].long()
    slots = torch.where((row < indptr[n]) & given[seq], block * page + t % page, -1)
    left = free - torch.where(given, need, 0).sum()
    return torch.where(given, old + new, old).int(), indptr.int(), slots, left.int()


def _plain_append(s):
    slots, page = s["slots"], s["page"]
    kept = slots >= 0
    block, place = slots[kept] // page, slots[kept] % page
    s["k_cache"][block, :, place] = s["k_new"][kept]
    s["v_cache"][block, :, place] = s["v_new"][kept]
    return s["k_cache"], s["v_cache"]


def _gather(cache, factor, table, tokens):
    """Rows of the first `tokens` tokens of each table row, [n, K, tokens, D] in 32 bits."""
    x = cache[table.long()]
    x = x.view(torch.float8_e4m3fn).float() * factor[table.long()][..., None] if factor is not None else x.float()
    return x.transpose(1, 2).flatten(2, 3)[:, :, :tokens]


def _scores(s, q, k, distance):
    """[n, K, rows, G, tokens]; q [n, rows, H, D], k [n, K, tokens, D], distance [n, rows, tokens]."""
    n, rows, H, D = q.shape
    K = k.shape[1]
    x = q.unflatten(2, (K, H // K)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    x = torch.matmul(x, k.transpose(2, 3)).unflatten(2, (rows, H // K))
    x *= s["scale"]
    if s["softcap"]:
        x = x.div_(s["softcap"]).tanh_().mul_(s["softcap"])
    if s["slopes"] is not None:
        x -= s["slopes"].view(1, K, 1, H // K, 1) * distance[:, None, :, None, :]
    return x


def _weigh(x, seen, v):
    """(max, sum, weighted V) of the seen tokens: [n, K, rows, G], the same, [n, K, rows, G, D]."""
    x = x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = x.sub_(top).exp_()
    o = torch.matmul(x.flatten(2, 3), v).unflatten(2, x.shape[2:4])
    return top.squeeze(-1), x.sum(-1), o


def _by_rows(o, total):
    """[n, K, rows, G, D] over the sums -> [n, rows, H, D]; a row that saw nothing is zero."""
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    return o.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attend(s):
    table = s["block_tables"]
    n = table.shape[0]
    k = _gather(s["k_cache"], s.get("k_scale"), table, s["most"])
    v = _gather(s["v_cache"], s.get("v_scale"), table, s["most"])
    seq, at = s["seq"], s["at"]
    q = torch.zeros(n, s["widest"], *s["q"].shape[1:], device="cuda")
    q[seq, at] = s["q"].float()
    length = s["seq_lens"].long()
    count = (s["qo_indptr"][1:] - s["qo_indptr"][:-1]).long()
    pos = (length - count)[:, None] + torch.arange(s["widest"], device="cuda")
    t = torch.arange(s["most"], device="cuda")
    seen = t >= 0
    if s["window"]:
        seen = seen & (t > (pos - s["window"])[..., None])
    if s["doc_starts"] is not None:
        start = torch.zeros_like(pos)
        start[seq, at] = s["doc_starts"].long()
        seen = seen & (t >= start[..., None])
    if s["causal"]:
        seen = seen & (t <= pos[..., None])
    if s["prefix_lens"] is not None:
        seen = seen | (t < s["prefix_lens"].long()[:, None, None])
    seen = seen & (t < length[:, None, None])
    distance = (pos[..., None] - t).abs().float() if s["slopes"] is not None else None
    x = _scores(s, q, k, distance)
    top, total, o = _weigh(x, seen, v)
    return _by_rows(o, total)[seq, at].to(torch.bfloat16)


def _plain_shared(s):
    group, member = s["group"], s["member"]
    pre, length = s["prefix_lens"].long(), s["seq_lens"].long()
    q = s["q"].float()
    qg = torch.zeros(len(pre), s["widest"], *q.shape[1:], device="cuda")
    qg[group, member] = q
    place = torch.zeros(len(pre), s["widest"], dtype=torch.int64, device="cuda")
    place[group, member] = pre[group] + length - 1
    t = torch.arange(s["most_prefix"], device="cuda")
    away = (place[..., None] - t).float() if s["slopes"] is not None else None
    x = _scores(s, qg, _gather(s["k_cache"], None, s["prefix_tables"], len(t)), away)
    seen = (t < pre[:, None, None]).expand(-1, s["widest"], -1)
    m1, l1, o1 = _weigh(x, seen, _gather(s["v_cache"], None, s["prefix_tables"], len(t)))
    m1, l1, o1 = (y[group, :, member].unsqueeze(2) for y in (m1, l1, o1))
    t = torch.arange(max(1, s["most"]), device="cuda")
    away = (length[:, None, None] - 1 - t).float() if s["slopes"] is not None else None
    x = _scores(s, q[:, None], _gather(s["k_cache"], None, s["block_tables"], len(t)), away)
    m2, l2, o2 = _weigh(x, t < length[:, None, None], _gather(s["v_cache"], None, s["block_tables"], len(t)))
    m = torch.maximum(m1, m2)
    a, b = (m1 - m).exp(), (m2 - m).exp()
    return _by_rows(o1 * a[..., None] + o2 * b[..., None], l1 * a + l2 * b)[:, 0].to(torch.bfloat16)


def _mods(s):
    return dict(softcap=s["softcap"], alibi_slopes=s["slopes"], window=s["window"],
                prefix_lens=s["prefix_lens"], doc_starts=s["doc_starts"])


def run(s):
    op = s["op"]
    if own:
        import paged_kv_gqa_decode_gb300 as pa
        if op == "assign":
            lens, indptr, slots, left = pa.paged_kv_assign(
                s["seq_lens"], s["new_lens"], s["block_tables"], s["free_blocks"], s["free_count"],
                s["page"], s["max_new"])
            return lens, indptr, slots, left, s["block_tables"]
        if op == "append":
            pa.paged_kv_append_slots(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["slots"])
            return s["k_cache"], s["v_cache"]
        if op == "shared":
            return pa.paged_attn_decode_shared(
                s["q"], s["k_cache"], s["v_cache"], s["group_indptr"], s["prefix_tables"],
                s["prefix_lens"], s["block_tables"], s["seq_lens"], s["scale"],
                softcap=s["softcap"], alibi_slopes=s["slopes"])
        if op == "multi":
            return pa.paged_attn_decode_multi_mods(
                s["q"], s["k_cache"], s["v_cache"], s["qo_indptr"], s["block_tables"],
                s["seq_lens"], s["scale"], causal=s["causal"], **_mods(s))
        if "k_scale" in s:
            return pa.paged_attn_decode_fp8_mods(
                s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_tables"],
                s["seq_lens"], s["scale"], **_mods(s))
        return pa.paged_attn_decode_mods(s["q"], s["k_cache"], s["v_cache"], s["block_tables"],
                                         s["seq_lens"], s["scale"], **_mods(s))
    if op == "assign":
        return (*_plain_assign(s), s["block_tables"])
    if op == "append":
        return _plain_append(s)
    return _plain_shared(s) if op == "shared" else _plain_attend(s)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    """One sequence at a time, over the tokens in their own order, in 64 bits."""
    if case["op"] in ("assign", "append"):
        return None  # whole numbers and copies
    s = prepare(case, seed)
    page, H, K = case["page"], case["heads"], case["kv_heads"]
    G = H // K

    def rows(name, ids, n):
        c = s[name + "_cache"][ids.long()]                       # [pages, K, page, D]
        if name + "_scale" in s:
            c = c.view(torch.float8_e4m3fn).double() * s[name + "_scale"][ids.long()].double()[..., None]
        return c.double().permute(0, 2, 1, 3).reshape(-1, K, c.shape[-1])[:n]

    def softmax_rows(q, k, v, seen, away):
        """q [r, D], k, v [t, D], seen [r, t], away [r, t] or None (per-head distance bias)."""
        x = (q @ k.T) * float(np.float32(s["scale"]))
        if s["softcap"]:
            x = s["softcap"] * torch.tanh(x / s["softcap"])
        if away is not None:
            x = x - away
        w = torch.softmax(torch.where(seen, x, -math.inf), dim=-1)
        return torch.where(seen.any(-1, keepdim=True), w, 0.0) @ v

    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lens = _lens(case)
    if case["op"] == "shared":
        pre = _spread(case["pre_lo"], case["pre_hi"], case["groups"], 4)
        group = np.repeat(np.arange(case["groups"]), _group_sizes(case))
        row_of = [[i] for i in range(len(lens))]
        total = pre[group] + lens
    else:
        seq, pos, lo, hi = _rows(case)
        row_of = [np.nonzero(seq == i)[0] for i in range(len(lens))]
        total = lens
        pre = _prefixes(case) if case["prefix"] else np.zeros_like(lens)
    held = None
    for i, n in enumerate(total):
        if n == 0 or not len(row_of[i]):
            continue
        own_pages = s["block_tables"][i, :-(-int(lens[i]) // page)]
        k, v = rows("k", own_pages, int(lens[i])), rows("v", own_pages, int(lens[i]))
        if case["op"] == "shared":
            g = int(group[i])
            if held is None or held[0] != g:
                ids = s["prefix_tables"][g, :-(-int(pre[g]) // page)]
                held = (g, rows("k", ids, int(pre[g])), rows("v", ids, int(pre[g])))
            k, v = torch.cat([held[1], k]), torch.cat([held[2], v])
        t = torch.arange(int(n), device="cuda")
        r = torch.tensor(row_of[i], device="cuda")
        if case["op"] == "shared":
            p = torch.tensor([int(n) - 1], device="cuda")
            seen = torch.ones(1, int(n), dtype=torch.bool, device="cuda")
        else:
            p, a, b = (torch.tensor(x[row_of[i]], device="cuda")[:, None] for x in (pos, lo, hi))
            seen = ((t >= a) & (t <= b)) | (t < int(pre[i]))
            p = p[:, 0]
        away = (p[:, None] - t).abs().double() if case["alibi"] else None
        for h in range(H):
            bias = away * float(s["slopes"][h]) if away is not None else None
            out[r, h] = softmax_rows(s["q"][r, h].double(), k[:, h // G], v[:, h // G], seen, bias)
    return out
