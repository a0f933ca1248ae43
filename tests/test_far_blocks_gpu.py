"""Blocks whose rows lie past 2^31 elements (and 2^32 bytes) of the cache: each operator gives the
bits that it gives on a small cache with the same rows."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_decode_gb300 as pa
from oracle import speculative as sp

pytestmark = pytest.mark.gpu

H, BS, D, SMALL, BIG = 8, 16, 256, 24, 70000
DEV = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def caches():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_decode_gb300 import build

    build.build()
    pa.load()
    g = torch.Generator(device="cuda").manual_seed(1)
    assert BIG * H * BS * D > 2 ** 31
    made = {}
    for fp8 in (False, True):
        big = [torch.empty(BIG, H, BS, D, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda") for _ in range(2)]
        rows = [torch.randn(SMALL, H, BS, D, generator=g, device="cuda") for _ in range(2)]
        rows = [r.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else r.to(torch.bfloat16) for r in rows]
        floats = [torch.rand(BIG, H, BS, device="cuda") for _ in range(2)] if fp8 else None
        made[fp8] = big, rows, floats
    return made


def both(caches, fp8, call):
    """call(first block, k, v, floats) on the small cache and at the end of the big one."""
    big, rows, floats = caches[fp8]
    outs = []
    for first in (0, BIG - SMALL):
        if first:
            for b, r in zip(big, rows):
                b[first:] = r
            k, v = big
            f = {} if floats is None else dict(k_scale=floats[0], v_scale=floats[1])
        else:
            k, v = (r.clone() for r in rows)
            f = {} if floats is None else dict(k_scale=floats[0][-SMALL:].clone(), v_scale=floats[1][-SMALL:].clone())
            if floats is not None:
                kept = [t.clone() for t in f.values()]
        out = call(first, k, v, f)
        torch.cuda.synchronize()
        outs.append([*out, k[-SMALL:].clone(), v[-SMALL:].clone(), *(t[-SMALL:].clone() for t in f.values())])
        if first == 0 and floats is not None:
            for t, old in zip(floats, kept):
                t[-SMALL:] = old
    for a, b in zip(*outs):
        assert torch.equal(a.view(torch.int16) if a.dtype is torch.bfloat16 else a,
                           b.view(torch.int16) if b.dtype is torch.bfloat16 else b)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [3, 900])
def test_rotation_and_append(caches, fp8, rows):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(rows, 4 * H * D, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([2 * H * D, H * D, H * D], 1))
    slots = torch.randperm(SMALL * BS, generator=g, device="cuda")
    slots = torch.cat([slots, torch.full((max(rows - SMALL * BS, 0),), -1, device="cuda")])[:rows]
    angle = torch.arange(50, device="cuda")[:, None] * torch.rand(D // 2, generator=g, device="cuda")
    cs = torch.cat([angle.cos(), angle.sin()], 1)
    pos = torch.arange(rows, **DEV) % 50
    both(caches, fp8, lambda first, kc, vc, f: [pa.paged_kv_rope_append_slots(
        q, k, v, kc, vc, torch.where(slots < 0, slots, slots + first * BS), pos, cs, **f)])


@pytest.mark.parametrize("fp8", [False, True])
def test_compaction_and_forks(caches, fp8):
    table = torch.arange(SMALL, **DEV).flip(0)[:20].reshape(4, 5).contiguous()
    lens, qo = torch.tensor([80, 77, 0, 0], **DEV), torch.tensor([0, 40, 77, 77, 77], **DEV)
    acc = torch.tensor([[1, 5, 6, 39], [0, 30, -1, -1], [-1] * 4, [-1] * 4], **DEV)

    def call(first, k, v, f):
        nb = k.shape[0]
        t = table + first
        kept = pa.paged_kv_compact(k, v, qo, acc, t, lens, **f)
        free = torch.arange(SMALL - 20, **DEV) + first
        left = pa.paged_kv_fork(k, v, t, kept, torch.tensor([0, 1], **DEV), torch.tensor([3, 2], **DEV),
                                torch.zeros(nb, **DEV), free, torch.tensor([SMALL - 20], **DEV), **f)
        return [kept, left, t - first]

    both(caches, fp8, call)


def test_trees(caches):
    table = torch.arange(SMALL, **DEV).flip(0).reshape(2, 12).contiguous()
    lens, ql = torch.tensor([190, 60], **DEV), [20, 33]
    rng = np.random.default_rng(3)
    bits = [np.tril(rng.random((m, m)) < 0.4) | np.eye(m, dtype=bool) for m in ql]
    mask = torch.tensor(np.concatenate([sp.mask_words(b, 2) for b in bits]), device="cuda")
    qo = torch.tensor([0, 20, 53], **DEV)
    q = torch.randn(53, 2 * H, D, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(torch.bfloat16)
    both(caches, False, lambda first, k, v, f: [pa.paged_attn_decode_tree(q, k, v, qo, mask, table + first, lens, 0.06)])
