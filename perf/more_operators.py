"""Cases of the operators of speculative and parallel decoding over the paged KV cache, with their plain forms.

Five operators, in the order in which an engine calls them around its attention:

* ``rope``    -- norms of each query and key head, their rotation by one or several axes of
  positions, and the append of the K and V rows by slot, to a bf16 or FP8 cache;
* ``tree``    -- attention of a tree of drafted tokens over the cache;
* ``compact`` -- the rows of the accepted drafted tokens moved together in the cache;
* ``fork``    -- sequences that continue another one: whole pages shared, the last one copied;
* ``release`` -- pages of finished sequences and dropped drafts back to the free stack.

``run`` computes an operator in elementary torch operations in 32 bits, or, when ``own`` is
true, through the framework's entry points.  A drafted row sees drafted token j of its
sequence where bit j of its mask is set, and cached token t when t < prefix or
t > pos - window, pos being the tokens before the tree plus the drafted ones it sees, less one.
"""
import math

import numpy as np
import torch

own = False

_LLAMA = dict(heads=32, kv_heads=8, dim=128)
_WIDE = dict(heads=24, kv_heads=4, dim=256)


def listed():
    return [
        # the rows of a decode step, slices of one fused projection, heads with norms
        dict(_LLAMA, name="rope_step", op="rope", rows=256, page=16, rot=128, axes=1, norm=True,
             inter=False, fp8=False),
        # a prefill step of text and images: time, height and width positions
        dict(_LLAMA, name="rope_prompts", op="rope", rows=8192, page=16, rot=128, axes=3, norm=True,
             inter=False, fp8=False),
        # an odd number of rows, a quarter of wide heads rotated in neighbouring pairs, FP8 caches
        dict(_WIDE, name="rope_fp8_wide", op="rope", rows=4001, page=16, rot=64, axes=1, norm=False,
             inter=True, fp8=True),
        # two short chats with a few drafts each in a capped, windowed layer: latency counts
        dict(name="tree_tiny", op="tree", heads=4, kv_heads=2, dim=64, page=16, seqs=2, len_lo=37,
             len_hi=100, q_lo=5, q_hi=9, softcap=30.0, window=64, prefix=4, alibi=False),
        # verification of trees of 16 to 64 drafted tokens
        dict(_LLAMA, name="tree_verify", op="tree", page=16, seqs=32, len_lo=512, len_hi=4096, q_lo=16,
             q_hi=64, softcap=0.0, window=0, prefix=0, alibi=False),
        # trees over four contexts of 100000 tokens, wide heads
        dict(_WIDE, name="tree_long", op="tree", page=16, seqs=4, len_lo=100000, len_hi=100000, q_lo=24,
             q_hi=41, softcap=0.0, window=0, prefix=0, alibi=False),
        # the accepted paths of that verification
        dict(_LLAMA, name="compact_step", op="compact", page=16, seqs=32, len_lo=512, len_hi=4096, q_lo=16,
             q_hi=64, depth=8, fp8=False),
        # long paths of a large batch, FP8 caches
        dict(_LLAMA, name="compact_fp8", op="compact", page=32, seqs=256, len_lo=200, len_hi=2000, q_lo=40,
             q_hi=64, depth=40, fp8=True),
        # beam search: four beams from each of sixteen contexts
        dict(_LLAMA, name="fork_beams", op="fork", page=16, parents=16, each=3, len_lo=512, len_hi=4096,
             fp8=False),
        # eight samples of each of 64 prompts
        dict(_LLAMA, name="fork_samples", op="fork", page=32, parents=64, each=8, len_lo=100, len_hi=4000,
             fp8=False),
        # the dropped drafts of a large batch
        dict(name="release_step", op="release", page=16, seqs=256, len_lo=100, len_hi=32768, share=1,
             cut=80, finished=0.02),
        # the end of many sequences that share prompts
        dict(name="release_finished", op="release", page=16, seqs=512, len_lo=100, len_hi=16384, share=4,
             cut=0, finished=0.6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "tree", "tree", "compact", "fork", "release"])
    page = rng.choice([16, 32])
    if op == "release":
        len_hi = _log(rng, 16, 32768)
        seqs = _log(rng, 1, max(2, min(1024, 8000000 // len_hi)))
        return dict(op=op, page=page, seqs=seqs, len_lo=rng.randint(0, min(100, len_hi)), len_hi=len_hi,
                    share=rng.choice([1, 1, 2, 5]), cut=rng.choice([0, _log(rng, 1, 500)]),
                    finished=rng.choice([0.0, 0.1, 0.5, 1.0]))
    kv_heads = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128, 256])
    shape = dict(kv_heads=kv_heads, heads=kv_heads * rng.choice([1, 2, 4, 5, 6, 8, 16]), dim=dim, page=page)
    fp8 = dim >= 128 and rng.random() < 0.4
    if op == "rope":
        most = 8192 * 48 * 128 // ((shape["heads"] + 2 * kv_heads) * dim)
        return dict(shape, op=op, rows=_log(rng, 1, min(8192, most)), rot=16 * rng.randint(1, dim // 16),
                    axes=rng.choice([1, 1, 2, 3]), norm=rng.random() < 0.6, inter=rng.random() < 0.4, fp8=fp8)
    if op == "tree":
        seqs = _log(rng, 1, 32)
        len_hi = min(100000, _log(rng, 64, max(65, 100000 * 16 * 256 // (seqs * kv_heads * dim))))
        room = 4e10 / (shape["heads"] * len_hi * seqs * dim)
        q_hi = max(1, min(_log(rng, 1, 128), int(room), len_hi))
        return dict(shape, op=op, seqs=seqs, len_lo=rng.randint(q_hi, len_hi) if q_hi < len_hi else len_hi,
                    len_hi=len_hi, q_lo=rng.randint(1, q_hi), q_hi=q_hi, softcap=rng.choice([0.0, 0.0, 30.0]),
                    window=rng.choice([0, 0, _log(rng, 16, 4096)]), prefix=rng.choice([0, 0, 4]),
                    alibi=rng.random() < 0.2)
    if op == "compact":
        seqs = _log(rng, 1, 256)
        q_hi = _log(rng, 1, 128)
        len_hi = max(q_hi, min(_log(rng, 64, 4096), 500000 * 8 * 128 // (seqs * kv_heads * dim)))
        return dict(shape, op=op, seqs=seqs, len_lo=q_hi, len_hi=len_hi, q_lo=rng.randint(1, q_hi), q_hi=q_hi,
                    depth=_log(rng, 1, q_hi), fp8=fp8)
    parents = _log(rng, 1, 64)
    len_hi = min(_log(rng, 16, 8192), 300000 * 8 * 128 // (parents * kv_heads * dim))
    return dict(shape, op=op, parents=parents, each=rng.randint(1, 8), len_lo=rng.randint(0, min(64, len_hi)),
                len_hi=len_hi, fp8=fp8)


# ------------------------------------------------------------------ sizes of a case

def _spread(lo, hi, n, seed):
    """n lengths from hi to lo, log-uniform between them; the same for every seed of a case."""
    rng = np.random.default_rng(seed)
    a = max(lo, 1)
    x = np.round(np.exp(rng.uniform(math.log(a), math.log(max(hi, a)), size=n))).astype(np.int64)
    x = np.clip(x, lo, hi)
    x[0] = hi
    if n > 1:
        x[-1] = lo
    return x


def _lens(case):
    return _spread(case["len_lo"], case["len_hi"], case["parents"] if case["op"] == "fork" else case["seqs"], 1)


def _q_lens(case):
    return np.minimum(_spread(case["q_lo"], case["q_hi"], case["seqs"], 2), _lens(case))


def _depths(case):
    """Accepted tokens of each sequence: none, the bound, and between."""
    ql = _q_lens(case)
    n = np.arange(len(ql)) * 7 % (case["depth"] + 1)
    return np.minimum(np.where(np.arange(len(ql)) == 0, case["depth"], n), ql)


def _keeps(case):
    lens = _lens(case)
    rng = np.random.default_rng(3)
    keep = np.maximum(lens - rng.integers(0, case["cut"] + 1, size=len(lens)), 0)
    return np.where(rng.random(len(lens)) < case["finished"], 0, keep)


def _pages(case, tokens):
    return -(-tokens // case["page"])


def _shared_pages(case):
    """Leading pages that the sequences of a group hold together."""
    pages = _pages(case, _lens(case))
    group = np.arange(len(pages)) // case["share"]
    least = np.full(group.max() + 1, 1 << 40)
    np.minimum.at(least, group, pages)
    return group, least[group] * 3 // 4 if case["share"] > 1 else np.zeros_like(pages)


def _row_bytes(case):
    return 2 * case["kv_heads"] * ((case["dim"] + 4) if case.get("fp8") else 2 * case["dim"])


def work(case):
    op = case["op"]
    if op == "release":
        cut = int((_pages(case, _lens(case)) - _pages(case, np.minimum(_keeps(case), _lens(case)))).sum())
        # an entry and a count in, a count and a free entry out; lengths in and out
        return {"bytes": float(cut * 16 + case["seqs"] * 12 + 8), "flops": 0.0}
    D, H, K = case["dim"], case["heads"], case["kv_heads"]
    if op == "rope":
        rows = case["rows"]
        table = min(rows, 4096) * case["rot"] * 4
        return {"bytes": float(rows * ((2 * H + 2 * K) * D * 2 + _row_bytes(case) + 8 + 4 * case["axes"]) + table),
                "flops": float(rows * (H + K) * D * 8)}
    lens = _lens(case)
    if op == "fork":
        full, tail = lens // case["page"], lens % case["page"]
        n = case["each"]
        # a tail read once, written for each child; table entries in and out, counts in and out
        return {"bytes": float(int(tail.sum()) * _row_bytes(case) * (1 + n) + int(full.sum()) * (12 + 4 * n)
                               + int((tail > 0).sum()) * 8 * n + len(lens) * n * 12), "flops": 0.0}
    ql = _q_lens(case)
    if op == "compact":
        moved = int(np.maximum(_depths(case) - 1, 0).sum())
        return {"bytes": float(moved * (2 * _row_bytes(case) + 4) + len(lens) * 16), "flops": 0.0}
    ctx = lens - ql
    depth = np.log2(ql + 1.0) + 1
    seen = ctx if not case["window"] else np.minimum(ctx, case["window"] + case["prefix"])
    pairs = float((ql * (seen + depth)).sum())
    return {"bytes": float(int((seen + ql).sum()) * K * 4 * D + int(ql.sum()) * (H * D * 4 + 8)
                           + int(_pages(case, seen).sum()) * 4),
            "flops": 4.0 * D * H * pairs}


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


def _caches(s, case, blocks, gen):
    shape = (blocks, case["kv_heads"], case["page"], case["dim"])
    k, v = _normal(shape, gen), _normal(shape, gen)
    if case.get("fp8"):
        s["k_cache"], s["k_scale"] = _to_fp8(k)
        s["v_cache"], s["v_scale"] = _to_fp8(v)
    else:
        s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = k, v, None, None


def _trees(rng, q_lens):
    """Ancestors of each drafted token, itself included: bool [seqs, widest, widest].  A token hangs from
    one of the few before it or from the cached tokens; every 13th is padding, which sees none and is seen by none."""
    n, w = len(q_lens), int(q_lens.max())
    seen = np.zeros((n, w, w), dtype=bool)
    rows = np.arange(n)
    pad = np.arange(w) % 13 == 12
    for j in range(w):
        parent = j - 1 - np.minimum(rng.geometric(0.4, size=n) - 1, 6)
        ok = (parent >= 0) & ~pad[np.maximum(parent, 0)]
        if not pad[j]:
            seen[:, j] = np.where(ok[:, None], seen[rows, np.maximum(parent, 0)], False)
            seen[:, j, j] = True
    inside = np.arange(w)[None, :] < q_lens[:, None]
    return seen & inside[:, :, None] & inside[:, None, :]


def _words(seen):
    """int32 words of the bits, [..., words]."""
    w = seen.shape[-1]
    words = -(-w // 32)
    bits = np.zeros((*seen.shape[:-1], words * 32), dtype=np.uint64)
    bits[..., :w] = seen
    x = (bits.reshape(*seen.shape[:-1], words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return x.astype(np.uint32).view(np.int32)


def _slopes(heads):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)],
                        dtype=torch.float32, device="cuda")


def _prepare_rope(s, case, rng, gen):
    rows, page, D, H, K, R = (case[x] for x in ("rows", "page", "dim", "heads", "kv_heads", "rot"))
    blocks = -(-rows // page) * 5 // 4 + 2
    _caches(s, case, blocks, gen)
    qkv = _normal((rows, (H + 2 * K) * D), gen, 1.5)  # a fused projection's output
    slots = rng.permutation(blocks * page)[:rows]
    slots[rng.random(rows) < 0.02] = -1               # padding rows of the step
    # a few prompts (their positions in order, each from a place of its own), images of 32 x 32 in them
    start = rng.integers(0, 28000, size=8)
    pos = (start[np.arange(rows) % 8] if rows < 512 else start[np.arange(rows) * 8 // rows]) + np.arange(rows) % 4096
    at = np.arange(rows) % 1024
    axes = np.stack([pos, pos // 4 + at // 32, pos // 4 + at % 32])[:case["axes"]]
    angle = torch.arange(32768, dtype=torch.float64, device="cuda")[:, None] * (
        10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R))
    s.update(q=qkv[:, :H * D].unflatten(1, (H, D)), k_new=qkv[:, H * D:(H + K) * D].unflatten(1, (K, D)),
             v_new=qkv[:, (H + K) * D:].unflatten(1, (K, D)),
             slots=torch.tensor(slots, dtype=torch.int64, device="cuda"),
             positions=_i32(axes if case["axes"] > 1 else axes[0]),
             freq_axis=_i32(np.arange(R // 2) * case["axes"] // (R // 2)) if case["axes"] > 1 else None,
             cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(), inter=case["inter"],
             q_norm=1 + 0.2 * torch.randn(D, generator=gen, device="cuda") if case["norm"] else None,
             k_norm=1 + 0.2 * torch.randn(D, generator=gen, device="cuda") if case["norm"] else None, eps=1e-6)


def _prepare_release(s, case, rng):
    lens, keep = _lens(case), _keeps(case)
    group, shared = _shared_pages(case)
    pages = _pages(case, lens)
    maxb = max(1, int(pages.max()) + 2)
    bt = _tables(rng, pages, 0, maxb)
    first = group * case["share"]
    together = np.arange(maxb)[None, :] < shared[:, None]
    bt = np.where(together, bt[first], bt)
    used = np.arange(maxb)[None, :] < pages[:, None]
    blocks = int(pages.sum()) + 50
    refs = np.bincount(bt[used], minlength=blocks) - 1
    free = 40  # blocks of the stack before the call; there is room for all of them
    stack = np.full(blocks, -1, dtype=np.int64)
    stack[:free] = int(pages.sum()) + 1 + np.arange(free)
    s.update(block_tables=_i32(bt), seq_lens=_i32(lens), keep_lens=_i32(keep), block_refs=_i32(np.maximum(refs, 0)),
             free_blocks=_i32(stack), free_count=_i32([free]))


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, page = case["op"], case["page"]
    s = {"op": op, "page": page}
    if op == "rope":
        _prepare_rope(s, case, rng, gen)
        return s
    if op == "release":
        _prepare_release(s, case, rng)
        return s
    lens = _lens(case)
    pages = _pages(case, lens)
    maxb = max(1, int(pages.max()))
    if op == "fork":
        n, kids = len(lens), len(lens) * case["each"]
        used = int(pages.sum())
        blocks = used + kids + 20
        rows = rng.permutation(n + kids)  # the table rows of parents and children, in any order
        bt = np.full((n + kids, maxb), used, dtype=np.int64)
        bt[rows[:n]] = _tables(rng, pages, 0, maxb)
        held = np.zeros(n + kids, dtype=np.int64)
        held[rows[:n]] = lens
        _caches(s, case, blocks, gen)
        s.update(block_tables=_i32(bt), seq_lens=_i32(held), parents=_i32(np.repeat(rows[:n], case["each"])),
                 children=_i32(rows[n:]), block_refs=_i32(np.zeros(blocks)),
                 free_blocks=_i32(used + 1 + rng.permutation(blocks - used - 1)), free_count=_i32([kids + 9]))
        return s
    ql = _q_lens(case)
    _caches(s, case, int(pages.sum()) + 1, gen)
    s.update(block_tables=_i32(_tables(rng, pages, 0, maxb)), seq_lens=_i32(lens),
             qo_indptr=_i32(np.concatenate([[0], np.cumsum(ql)])))
    if op == "compact":
        accepted = np.full((len(ql), case["depth"]), -1, dtype=np.int64)
        for i, n in enumerate(_depths(case)):
            accepted[i, :n] = np.sort(rng.permutation(ql[i])[:n])
        s["accepted"] = _i32(accepted)
        return s
    D, H = case["dim"], case["heads"]
    seen = _trees(rng, ql)
    seq = np.repeat(np.arange(len(ql)), ql)
    at = np.arange(len(seq)) - np.repeat(np.cumsum(ql) - ql, ql)
    s.update(scale=1.0 / math.sqrt(D), softcap=float(case["softcap"]), window=case["window"], heads=H,
             slopes=_slopes(H) if case["alibi"] else None, most=int(lens.max()),
             prefix_lens=_i32(np.minimum(lens - ql, case["prefix"] + np.arange(len(lens)) % 3))
             if case["prefix"] else None,
             tree_mask=_i32(_words(seen[seq, at])), seq=torch.tensor(seq, device="cuda"),
             at=torch.tensor(at, device="cuda"), widest=int(ql.max()), q=_normal((len(seq), H, D), gen))
    return s


# ------------------------------------------------------------------ the plain forms

def _rotated(s, x, norm):
    """[rows, heads, D] in 32 bits: the norm of each head, then the rotation of its first elements."""
    x = x.float()
    if norm is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * norm
    half = s["cos_sin"].shape[1] // 2
    pos = s["positions"].long()
    i = torch.arange(half, device="cuda")
    place = pos[:, None] if s["freq_axis"] is None else pos[s["freq_axis"].long()].T
    c, w = (s["cos_sin"][place, i + off][:, None] for off in (0, half))
    if s["inter"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * c - b * w, b * c + a * w], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * c - b * w, b * c + a * w], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _cache_outputs(s):
    if s["k_scale"] is None:
        return s["k_cache"], s["v_cache"]
    e4m3 = torch.float8_e4m3fn
    return s["k_cache"].view(e4m3), s["v_cache"].view(e4m3), s["k_scale"], s["v_scale"]


def _plain_rope(s):
    kept = s["slots"] >= 0
    block, place = s["slots"][kept] // s["page"], s["slots"][kept] % s["page"]
    k, v = _rotated(s, s["k_new"], s["k_norm"])[kept], s["v_new"][kept]
    if s["k_scale"] is not None:
        s["k_cache"][block, :, place], s["k_scale"][block, :, place] = _to_fp8(k)
        s["v_cache"][block, :, place], s["v_scale"][block, :, place] = _to_fp8(v)
    else:
        s["k_cache"][block, :, place] = k.to(torch.bfloat16)
        s["v_cache"][block, :, place] = v
    return (_rotated(s, s["q"], s["q_norm"]).to(torch.bfloat16), *_cache_outputs(s))


def _plain_tree(s):
    table, most = s["block_tables"].long(), s["most"]
    k, v = (s[c][table].float().transpose(1, 2).flatten(2, 3)[:, :, :most] for c in ("k_cache", "v_cache"))
    n, K = k.shape[:2]
    H, rows = s["heads"], s["widest"]
    seq, at = s["seq"], s["at"]
    q = torch.zeros(n, rows, *s["q"].shape[1:], device="cuda")
    q[seq, at] = s["q"].float()
    length = s["seq_lens"].long()
    count = (s["qo_indptr"][1:] - s["qo_indptr"][:-1]).long()
    ctx = (length - count)[:, None]
    j = torch.arange(rows, device="cuda")
    bits = torch.zeros(n, rows, rows, dtype=torch.bool, device="cuda")
    bits[seq, at] = (s["tree_mask"][:, j // 32] >> (j % 32) & 1).bool()
    pos = ctx + bits.sum(-1) - 1
    t = torch.arange(most, device="cuda")
    cached = t < ctx[..., None]
    if s["window"]:
        cached = cached & (t > (pos - s["window"])[..., None])
    if s["prefix_lens"] is not None:
        cached = cached | ((t < s["prefix_lens"].long()[:, None, None]) & (t < ctx[..., None]))
    draft = (t - ctx).clamp(0, rows - 1)
    drafted = (t >= ctx) & (t < length[:, None])
    seen = cached.expand(-1, rows, -1) | (bits.gather(2, draft[:, None].expand(-1, rows, -1)) & drafted[:, None])
    x = torch.matmul(q.unflatten(2, (K, H // K)).permute(0, 2, 1, 3, 4).flatten(2, 3), k.transpose(2, 3))
    x = x.mul_(s["scale"]).unflatten(2, (rows, H // K))
    if s["softcap"]:
        x = x.div_(s["softcap"]).tanh_().mul_(s["softcap"])
    if s["slopes"] is not None:
        at_t = torch.where(t < ctx, t, pos.gather(1, draft))
        away = (pos[..., None] - at_t[:, None]).abs().float()
        x -= s["slopes"].view(1, K, 1, H // K, 1) * away[:, None, :, None, :]
    x = x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1)
    o = torch.matmul(x.flatten(2, 3), v).unflatten(2, (rows, H // K))
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    return o.permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, at].to(torch.bfloat16)


def _plain_compact(s):
    """Entry i of a sequence counts while each entry up to it is past the one before and inside the tree."""
    acc = s["accepted"].long()
    count = (s["qo_indptr"][1:] - s["qo_indptr"][:-1]).long()[:, None]
    before = torch.cat([torch.full_like(acc[:, :1], -1), acc[:, :-1]], 1)
    good = ((acc > before) & (acc < count)).long().cumprod(1).bool()
    ctx = s["seq_lens"].long()[:, None] - count
    i = torch.arange(acc.shape[1], device="cuda")
    seq = torch.arange(acc.shape[0], device="cuda")[:, None].expand_as(acc)[good]
    src, dst, page = (ctx + acc)[good], (ctx + i)[good], s["page"]
    from_, to = (s["block_tables"][seq, x // page].long() for x in (src, dst))
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        if s[name] is not None:
            s[name][to, :, dst % page] = s[name][from_, :, src % page]
    return ((ctx[:, 0] + good.sum(1)).int(), *_cache_outputs(s))


def _plain_fork(s):
    """The last page's rows go to a block from the top of the free stack, fork by fork; a child whose block is
    not there stays empty."""
    page, bt, lens, refs = s["page"], s["block_tables"], s["seq_lens"], s["block_refs"]
    p, c = s["parents"].long(), s["children"].long()
    length = lens[p].long()
    full, tail = length // page, length % page
    free = s["free_count"].long()
    rank = (tail > 0).long().cumsum(0)
    given = (tail == 0) | (rank <= free)
    column = torch.arange(bt.shape[1], device="cuda")[None, :]
    whole = (column < full[:, None]) & given[:, None]
    ids = bt[p].long()
    refs.index_add_(0, ids[whole], torch.ones_like(ids[whole], dtype=torch.int32))
    part = given & (tail > 0)
    fresh = s["free_blocks"][(free - rank).clamp(min=0)].long()
    entry = torch.where(whole, ids, bt[c].long())
    entry = torch.where((column == full[:, None]) & part[:, None], fresh[:, None], entry)
    bt[c] = entry.int()
    lens[c] = torch.where(given, length, 0).int()
    src, dst, n = ids[part, full[part]], fresh[part], tail[part]
    row = torch.arange(page, device="cuda") < n[:, None]
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        if s[name] is not None:
            x = s[name]
            keep = row[:, None, :].reshape(len(n), 1, page, *[1] * (x.dim() - 3))
            x[dst] = torch.where(keep, x[src], x[dst])
    return bt, lens, refs, (free - part.sum()).int(), *_cache_outputs(s)


def _plain_release(s):
    """Each page past a sequence's kept tokens loses a holder; one that nobody holds any more goes to the top of
    the free stack, in the order of the sequences and pages (the first of several holders counts)."""
    bt, refs, page = s["block_tables"], s["block_refs"], s["page"]
    length = s["seq_lens"].long()
    keep = torch.minimum(s["keep_lens"].long(), length)
    column = torch.arange(bt.shape[1], device="cuda")[None, :]
    gone = (column >= ((keep + page - 1) // page)[:, None]) & (column < ((length + page - 1) // page)[:, None])
    ids = bt[gone].long()
    refs.index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
    order = torch.arange(len(ids), device="cuda")
    first = torch.full(refs.shape, len(ids), dtype=torch.int64, device="cuda").scatter_reduce_(0, ids, order, "amin")
    freed = ids[(refs[ids] < 0) & (first[ids] == order)]
    stack, free = s["free_blocks"], s["free_count"].long()
    stack[free + torch.arange(len(freed), device="cuda")] = freed.int()
    refs.clamp_(min=0)
    return keep.int(), refs, stack, (free + len(freed)).int()


def run(s):
    op = s["op"]
    if own:
        import paged_kv_gqa_decode_gb300 as pa
        if op == "rope":
            q = pa.paged_kv_rope_append_slots(
                s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["slots"], s["positions"],
                s["cos_sin"], freq_axis=s["freq_axis"], interleaved=s["inter"], q_norm=s["q_norm"],
                k_norm=s["k_norm"], eps=s["eps"], k_scale=s["k_scale"], v_scale=s["v_scale"])
            return (q, *_cache_outputs(s))
        if op == "tree":
            return pa.paged_attn_decode_tree(
                s["q"], s["k_cache"], s["v_cache"], s["qo_indptr"], s["tree_mask"], s["block_tables"],
                s["seq_lens"], s["scale"], softcap=s["softcap"], alibi_slopes=s["slopes"], window=s["window"],
                prefix_lens=s["prefix_lens"])
        if op == "compact":
            lens = pa.paged_kv_compact(s["k_cache"], s["v_cache"], s["qo_indptr"], s["accepted"],
                                       s["block_tables"], s["seq_lens"], k_scale=s["k_scale"],
                                       v_scale=s["v_scale"])
            return (lens, *_cache_outputs(s))
        if op == "fork":
            left = pa.paged_kv_fork(s["k_cache"], s["v_cache"], s["block_tables"], s["seq_lens"], s["parents"],
                                    s["children"], s["block_refs"], s["free_blocks"], s["free_count"],
                                    k_scale=s["k_scale"], v_scale=s["v_scale"])
            return s["block_tables"], s["seq_lens"], s["block_refs"], left, *_cache_outputs(s)
        lens, count = pa.paged_kv_release(s["block_tables"], s["seq_lens"], s["keep_lens"], s["free_blocks"],
                                          s["free_count"], s["page"], block_refs=s["block_refs"])
        return lens, s["block_refs"], s["free_blocks"], count
    return {"rope": _plain_rope, "tree": _plain_tree, "compact": _plain_compact, "fork": _plain_fork,
            "release": _plain_release}[op](s)


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_rope(case, s):
    D, R, page = case["dim"], case["rot"], case["page"]
    rows = case["rows"]
    pos = s["positions"].reshape(-1, rows).double()
    pair = torch.arange(R // 2, device="cuda")
    axis = (pair * case["axes"] // (R // 2)) if case["axes"] > 1 else torch.zeros_like(pair)
    at = pos[axis].long()                                            # [R / 2, rows]
    cs = s["cos_sin"].double()
    z = torch.complex(cs[at, pair[:, None]], cs[at, R // 2 + pair[:, None]]).T[:, None]

    def turn(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        out = x.clone()
        if case["inter"]:
            y = torch.complex(x[..., 0:R:2].contiguous(), x[..., 1:R:2].contiguous()) * z
            out[..., 0:R:2], out[..., 1:R:2] = y.real, y.imag
        else:
            y = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * z
            out[..., :R // 2], out[..., R // 2:R] = y.real, y.imag
        return out

    caches, floats = [], []
    for new, w, name in ((s["k_new"], s["k_norm"], "k"), (s["v_new"], None, "v")):
        x = turn(new, w) if name == "k" else new.double()
        cache = s[name + "_cache"]
        cache = (cache.view(torch.float8_e4m3fn) if case["fp8"] else cache).double()
        rows_of = cache.transpose(1, 2).reshape(-1, case["kv_heads"], D)
        to = s["slots"][s["slots"] >= 0]
        x = x[s["slots"] >= 0]
        if case["fp8"]:
            f = x.abs().amax(-1) / 448
            scale = s[name + "_scale"].double().transpose(1, 2).reshape(-1, case["kv_heads"])
            scale[to] = f
            floats.append(scale.reshape(-1, page, case["kv_heads"]).transpose(1, 2).contiguous())
            x = x / f[..., None]
        rows_of[to] = x
        caches.append(rows_of.reshape(-1, page, case["kv_heads"], D).transpose(1, 2).contiguous())
    return (turn(s["q"], s["q_norm"]), *caches, *floats)


def _exact_tree(case, s):
    """One sequence and head at a time, over the tokens in their own order."""
    page, H, K = case["page"], case["heads"], case["kv_heads"]
    lens, ql = _lens(case), _q_lens(case)
    words = s["tree_mask"].cpu().numpy().view(np.uint32)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for i, n in enumerate(int(x) for x in lens):
        m = int(ql[i])
        base = n - m
        ids = s["block_tables"][i, :-(-n // page)].long()
        see = np.array([[(int(words[row + a, b // 32]) >> (b % 32)) & 1 for b in range(m)] for a in range(m)], dtype=bool)
        place = base + see.sum(1) - 1
        t = np.arange(base)
        old = np.ones((m, base), dtype=bool)
        if case["window"]:
            old &= t[None, :] > place[:, None] - case["window"]
        if s["prefix_lens"] is not None:
            old |= t[None, :] < int(s["prefix_lens"][i])
        mask = torch.tensor(np.concatenate([old, see], 1), device="cuda")
        where = torch.tensor(np.concatenate([t, place]), device="cuda")
        away = (torch.tensor(place, device="cuda")[:, None] - where[None, :]).abs().double()
        for g in range(K):
            k, v = (s[c][ids, g].reshape(-1, case["dim"])[:n].double() for c in ("k_cache", "v_cache"))
            for h in range(g * (H // K), (g + 1) * (H // K)):
                x = s["q"][row:row + m, h].double() @ k.T * float(np.float32(s["scale"]))
                if s["softcap"]:
                    x = s["softcap"] * torch.tanh(x / s["softcap"])
                if s["slopes"] is not None:
                    x = x - float(s["slopes"][h]) * away
                w = torch.softmax(torch.where(mask, x, -math.inf), -1)
                out[row:row + m, h] = torch.where(mask.any(-1, keepdim=True), w, 0.0) @ v
        row += m
    return out


def exact(case, seed):
    if case["op"] not in ("rope", "tree"):
        return None  # whole numbers and copies
    s = prepare(case, seed)
    return _exact_rope(case, s) if case["op"] == "rope" else _exact_tree(case, s)
