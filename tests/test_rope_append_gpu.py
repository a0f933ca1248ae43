"""Norm, rotation and append in one pass against the float64 definition, element by element
within the roundings' bound."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_decode_gb300 as pa
from oracle import serving, speculative as sp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_decode_gb300 import build

    build.build()
    pa.load()


def table(most, R):
    angle = np.arange(most)[:, None] * 1000.0 ** (-np.arange(R // 2) / max(1, R // 2))
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def rows_of(cache, slots, BS):
    return cache[slots // BS, :, slots % BS]


def run_case(rows, H_q, H_kv, D, BS, R, seed=0, axes=1, sections=None, norm=True, inter=False, fp8=False,
             gap=0, most=200, eps=1e-5, scale=1.0, out_of_range=False, in_place=False, dense=False):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = (H_q + 2 * H_kv) * D + gap
    x = (torch.randn(rows, width, generator=g, device="cuda") * scale).to(torch.bfloat16)
    q, k, v = x[:, :H_q * D], x[:, H_q * D:(H_q + H_kv) * D], x[:, (H_q + H_kv) * D:(H_q + 2 * H_kv) * D]
    q, k, v = q.unflatten(1, (H_q, D)), k.unflatten(1, (H_kv, D)), v.unflatten(1, (H_kv, D))
    if dense:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    nb = -(-rows // BS) + 3
    slots = rng.permutation(nb * BS)[:rows]
    slots[rng.random(rows) < 0.1] = -1
    if rows > 3:
        slots[1] = nb * BS  # past the pool: not written
    pos = rng.integers(0, most, size=(axes, rows))
    if out_of_range:
        pos[0, ::3] = -5
        pos[-1, 1::3] = most + 9
    if sections is None:
        freq = np.arange(R // 2) * axes // max(1, R // 2)
    else:
        freq = np.asarray(sections)
    cs = table(most, R)
    wq, wk = (torch.randn(D, generator=g, device="cuda") if norm else None for _ in range(2))
    shape = (nb, H_kv, BS, D)
    if fp8:
        kc, vc = (torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2))
        kf, vf = (torch.full(shape[:3], 7.0, device="cuda") for _ in range(2))
    else:
        kc, vc = (torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        kf = vf = None
    hq, hk, hv = (serving.bf16_to_f64(t) for t in (q, k, v))
    d_slots = torch.tensor(slots, device="cuda")
    d_pos = torch.tensor(pos if axes > 1 else pos[0], dtype=torch.int32, device="cuda")
    out = pa.paged_kv_rope_append_slots(
        q, k, v, kc, vc, d_slots, d_pos, torch.tensor(cs).cuda(), interleaved=inter,
        freq_axis=torch.tensor(freq, dtype=torch.int32, device="cuda") if axes > 1 or sections is not None else None,
        q_norm=wq, k_norm=wk, eps=eps, k_scale=kf, v_scale=vf, out=q if in_place else None)
    torch.cuda.synchronize()
    host = lambda t: None if t is None else t.double().cpu().numpy()
    eps = float(np.float32(eps))
    z, err = sp.turn(hq, host(wq), eps, pos, freq, cs, inter)
    tol = err + serving.BF16_STEP * (np.abs(z) + err) + 1e-38
    assert (np.abs(serving.bf16_to_f64(out) - z) <= tol).all()
    kept = (slots >= 0) & (slots < nb * BS)
    to = slots[kept]
    z, err = sp.turn(hk, host(wk), eps, pos, freq, cs, inter)
    z, err = z[kept], err[kept]
    untouched = np.ones(nb * BS, dtype=bool)
    untouched[to] = False
    left = np.nonzero(untouched)[0]
    if not fp8:
        got_k, got_v = serving.bf16_to_f64(kc), serving.bf16_to_f64(vc)
        assert (np.abs(rows_of(got_k, to, BS) - z) <= err + serving.BF16_STEP * (np.abs(z) + err) + 1e-38).all()
        assert (rows_of(got_v, to, BS) == hv[kept]).all()
        assert (rows_of(got_k, left, BS) == 7).all() and (rows_of(got_v, left, BS) == 7).all()
        return
    f = rows_of(kf.cpu().numpy().astype(np.float64), to, BS)
    top = np.abs(z).max(-1)
    spread = err.max(-1)
    assert (np.abs(f - np.where(top > 0, top / 448, 1)) <= spread / 448 + 2 * sp.F32_STEP * f).all()
    got = rows_of(kc.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64), to, BS) * f[..., None]
    # half an e4m3 step of the value, half the smallest step below the normal range, the
    # float32 error of the value and (through f) of the quotient
    tol = sp.E4M3_STEP * (np.abs(z) + err) + f[..., None] * 2.0 ** -10 + err + 4 * sp.F32_STEP * np.abs(z)
    assert (np.abs(got - z) <= tol * (1 + 1e-6)).all()
    assert (rows_of(kc.cpu().numpy(), left, BS) == 0x7f).all() and (rows_of(vf.cpu().numpy(), left, BS) == 7).all()
    # V: the bytes and floats of the FP8 append
    n = len(to)
    k8, v8 = torch.zeros_like(kc), torch.zeros_like(vc)
    ks, vs = torch.zeros_like(kf), torch.zeros_like(vf)
    i32 = dict(dtype=torch.int32, device="cuda")
    bt = torch.tensor(to // BS, **i32)[:, None].contiguous()
    vd = v[torch.tensor(kept, device="cuda")].contiguous()
    pa.paged_kv_append_fp8(vd, vd, k8, v8, ks, vs, bt, torch.tensor(to % BS + 1, **i32))
    torch.cuda.synchronize()
    assert np.array_equal(rows_of(vc.cpu().numpy(), to, BS), rows_of(v8.cpu().numpy(), to, BS))
    assert np.array_equal(rows_of(vf.cpu().numpy(), to, BS), rows_of(vs.cpu().numpy(), to, BS))


@pytest.mark.parametrize("D,BS", [(64, 16), (128, 16), (128, 32), (256, 16)])
@pytest.mark.parametrize("rows,H_q,H_kv", [(1, 1, 1), (2, 4, 2), (5, 6, 3), (33, 5, 5), (300, 16, 1), (701, 24, 4)])
@pytest.mark.parametrize("inter", [False, True])
def test_shapes(D, BS, rows, H_q, H_kv, inter):
    run_case(rows, H_q, H_kv, D, BS, D, seed=rows, inter=inter)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("part", [0, 16, 48, -16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_parts_of_a_head_that_turn(D, part, inter, norm):
    run_case(37, 8, 2, D, 16, D + part if part < 0 else part, seed=D + part, inter=inter, norm=norm)


@pytest.mark.parametrize("D,BS", [(128, 16), (128, 32), (256, 32)])
@pytest.mark.parametrize("rows,H_q,H_kv", [(1, 4, 1), (45, 6, 2), (513, 10, 5)])
@pytest.mark.parametrize("inter", [False, True])
def test_fp8_caches(D, BS, rows, H_q, H_kv, inter):
    run_case(rows, H_q, H_kv, D, BS, D // 2, seed=rows, inter=inter, fp8=True, norm=rows != 45)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D", [128, 256])
def test_several_axes(D, inter, fp8):
    half = D // 2
    run_case(70, 8, 2, D, 16, D, axes=3, inter=inter, fp8=fp8, seed=1)
    run_case(70, 8, 2, D, 16, D, axes=3, sections=np.arange(half) % 3, inter=inter, fp8=fp8, seed=2)
    uneven = np.repeat([0, 1, 2], [half // 4, half // 8 + 5, half - half // 4 - half // 8 - 5])
    run_case(70, 8, 2, D, 16, D, axes=3, sections=uneven, inter=inter, fp8=fp8, seed=3)
    run_case(20, 8, 2, D, 16, D, axes=2, sections=np.arange(half) - 3, inter=inter, fp8=fp8, seed=4)  # clamped


# enough rows for the kernel that streams them
@pytest.mark.parametrize("rows,H_q,H_kv,D,kw", [
    (2601, 32, 8, 64, dict()), (2601, 40, 8, 64, dict(inter=True, axes=3)), (1501, 32, 8, 128, dict()),
    (1501, 32, 8, 128, dict(inter=True, norm=False)), (1501, 20, 10, 128, dict(fp8=True)),
    (1000, 32, 2, 128, dict(part=48, gap=8)), (1000, 33, 11, 128, dict(fp8=True, inter=True, part=64)),
    (701, 24, 4, 256, dict(fp8=True, part=64)), (801, 24, 4, 256, dict(axes=3)),
    (1501, 32, 8, 128, dict(axes=3, inter=False, mixed=True)), (1501, 32, 8, 128, dict(axes=2, fp8=True, mixed=True)),
    (1501, 32, 8, 128, dict(dense=True, in_place=True)), (1501, 32, 8, 128, dict(part=0)),
])
def test_many_rows(rows, H_q, H_kv, D, kw):
    kw = dict(kw)
    R = kw.pop("part", D)
    if kw.pop("mixed", False):
        kw["sections"] = np.arange(R // 2) % kw["axes"]
    run_case(rows, H_q, H_kv, D, 16, R, seed=rows, out_of_range=rows == 1000, **kw)


def test_positions_outside_the_table_are_clamped():
    run_case(50, 8, 2, 128, 16, 128, out_of_range=True)
    run_case(50, 8, 2, 128, 16, 128, axes=3, out_of_range=True, sections=np.arange(64) % 3)


def test_strides_and_queries_in_place():
    run_case(50, 8, 2, 128, 16, 128, gap=24)
    run_case(50, 8, 2, 128, 16, 64, dense=True, in_place=True)
    run_case(1, 8, 2, 64, 16, 64, in_place=True)


@pytest.mark.parametrize("at", ["before", "behind", "between"])
def test_queries_out_next_to_the_inputs(at):
    """Directly before, behind and between the rows of a projection that lie far apart."""
    rows, H_q, H_kv, D = 3, 2, 1, 64
    width, size = (H_q + 2 * H_kv) * D, rows * H_q * D
    stride = width + size if at == "between" else width + 8
    x = torch.randn(2 * size + rows * stride, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    fused = x[size:size + rows * stride].view(rows, stride)
    last = size + (rows - 1) * stride + width
    at = {"before": 0, "behind": last, "between": size + width}[at]
    out = x[at:at + size].view(rows, H_q, D)
    a, b = H_q * D, (H_q + H_kv) * D
    q, k, v = (t.unflatten(1, (-1, D)) for t in (fused[:, :a], fused[:, a:b], fused[:, b:width]))
    slots, pos = torch.arange(rows, device="cuda"), torch.arange(rows, dtype=torch.int32, device="cuda")
    cs = torch.tensor(table(8, D)).cuda()
    want = None
    for o in (None, out):
        kc, vc = (torch.zeros(1, H_kv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        got = (pa.paged_kv_rope_append_slots(q, k, v, kc, vc, slots, pos, cs, out=o), kc, vc)
        assert want is None or all(torch.equal(s, t) for s, t in zip(got, want))
        want = got
    with pytest.raises(pa.PagedAttnError):
        pa.paged_kv_rope_append_slots(q, k, v, kc, vc, slots, pos, cs, out=x[size + 8:][:size].view(rows, H_q, D))


@pytest.mark.parametrize("H_q,H_kv", [(4, 1), (8, 2), (3, 3)])
def test_few_heads_in_many_rows_of_fp8_caches(H_q, H_kv):
    run_case(2500, H_q, H_kv, 128, 16, 96, seed=H_q, fp8=True)


def test_small_and_large_values():
    run_case(20, 4, 2, 128, 16, 128, scale=1e-18, eps=0.0)
    run_case(20, 4, 2, 128, 16, 128, scale=1e15)
    run_case(20, 4, 2, 128, 16, 128, scale=1e-3, eps=1.0)
    run_case(20, 4, 2, 128, 16, 128, scale=1e4, norm=False, fp8=True)


def test_zero_rows_and_infinities():
    """A zero row stays zero (FP8: float 1); what does not turn keeps its infinity."""
    D, i32 = 128, dict(dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 1, D, dtype=torch.bfloat16, device="cuda")
    q[1, 0, 100] = float("inf")
    slots = torch.tensor([0, 1], device="cuda")
    cs = torch.tensor(table(10, 64)).cuda()
    kc, vc = (torch.full((1, 1, 16, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = pa.paged_kv_rope_append_slots(q, q, q, kc, vc, slots, torch.tensor([3, 4], **i32), cs, interleaved=False)
    assert torch.equal(out, q) and torch.equal(kc[0, :, :2], q.transpose(0, 1)) and torch.equal(vc[0, :, :2], q.transpose(0, 1))
    k8, v8 = (torch.full((1, 1, 16, D), 3, dtype=torch.uint8, device="cuda") for _ in range(2))
    kf, vf = (torch.zeros(1, 1, 16, device="cuda") for _ in range(2))
    w = torch.ones(D, device="cuda")
    pa.paged_kv_rope_append_slots(q[:1], q[:1], q[:1], k8, v8, slots[:1], torch.tensor([3], **i32), cs, k_norm=w,
                                  k_scale=kf, v_scale=vf)
    # (0 cos - 0 sin is minus zero where the cosine is negative)
    assert (k8[0, 0, 0] & 0x7f == 0).all() and (v8[0, 0, 0] == 0).all() and kf[0, 0, 0] == 1 and vf[0, 0, 0] == 1


def test_checks_report_slots_and_positions():
    D, i32 = 128, dict(dtype=torch.int32, device="cuda")
    q = torch.ones(3, 2, D, dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.zeros(2, 2, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cs = torch.tensor(table(10, 64)).cuda()
    for slots, pos, want in (([0, 1, -1], [0, 9, 5], 0), ([0, 32, 1], [0, 1, 2], 1), ([0, 1, 2], [0, 10, 2], 2),
                             ([40, 1, 2], [0, -1, 2], 3)):
        status = torch.zeros(1, **i32)
        try:
            pa.paged_attn_set_checks(2, status)
            pa.paged_kv_rope_append_slots(q, q, q, kc, vc, torch.tensor(slots, device="cuda"), torch.tensor(pos, **i32), cs)
        finally:
            pa.paged_attn_set_checks(0, None)
        assert int(status) == want


def test_no_rows():
    e = torch.zeros(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16, device="cuda")
    out = pa.paged_kv_rope_append_slots(e, e, e, kc, kc.clone(), torch.zeros(0, dtype=torch.int64, device="cuda"),
                                        torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(4, 128, device="cuda"))
    assert out.shape == (0, 2, 128)


def test_small_tensors_may_be_pinned_rows_and_caches_not():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 12, 128, generator=g).to(torch.bfloat16)
    q, k, v = (t.cuda() for t in (x[:, :8].contiguous(), x[:, 8:10].contiguous(), x[:, 10:].contiguous()))
    slots, pos = torch.tensor([3, 40, 0, -1, 9, 17]), torch.arange(6, dtype=torch.int32)
    cs = torch.tensor(table(8, 128))
    want = None
    for pinned in (False, True):
        kc, vc = (torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        s, p, t = (y.pin_memory() if pinned else y.cuda() for y in (slots, pos, cs))
        got = (pa.paged_kv_rope_append_slots(q, k, v, kc, vc, s, p, t), kc, vc)
        torch.cuda.synchronize()
        assert want is None or all(torch.equal(a, b) for a, b in zip(got, want))
        want = got
    host = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16).pin_memory()
    for bad in ((q.cpu().pin_memory(), k, v, kc, vc), (q, k.cpu().pin_memory(), v, kc, vc), (q, k, v, host, vc),
                (q, k, v, kc, host)):
        with pytest.raises(ValueError, match="device memory"):
            pa.paged_kv_rope_append_slots(*bad, slots.cuda(), pos.cuda(), cs.cuda())
