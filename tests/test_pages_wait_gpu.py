"""The bounded waits of the forks' and the rotation's copies, made to run out on purpose: in a test build of the library
(``build.build_wait_test``, waits of a few milliseconds, never part of the product) two pages' first copies are
waited for and never issued, or a row's queries are.  The launch reports status bit 2, the warps that waited copy nothing more, and
everything else is done.  Nothing here faults, traps or hangs: every wait that runs out returns."""
import ctypes

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_decode_gb300 import build
    import paged_kv_gqa_decode_gb300 as pa

    build.build()
    pa.load()
    x = ctypes.CDLL(build.build_wait_test())
    P, I, LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
    x.paged_kv_fork.argtypes = [P] * 13 + [I] * 7 + [LL, P]
    x.paged_attn_set_checks.argtypes = [LL, P]
    x.paged_attn_test_set_fork_fault.argtypes = [LL]
    x.paged_attn_test_set_rope_fault.argtypes = [LL]
    x.paged_kv_rope_append_slots.argtypes = ([P, P, P, LL, LL, LL] + [P] * 7 + [I, P, P] + [I, I, I, P, P, ctypes.c_float] +
                                             [I] * 5 + [LL, P])
    yield x
    x.paged_attn_test_set_fork_fault(-1)
    x.paged_attn_test_set_rope_fault(-1)
    x.paged_attn_set_checks(0, None)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def test_a_copy_that_does_not_come_is_reported(lib):
    forks, H, BS, D, tail = 700, 8, 32, 128, 31
    nb = forks + 2
    g = torch.Generator(device="cuda").manual_seed(1)
    first = torch.randn(nb, H, BS, D, generator=g, device="cuda").to(torch.bfloat16)
    k, v = first.clone(), first.clone()
    bt = torch.full((forks + 1, 2), -7, dtype=torch.int32, device="cuda")
    bt[0] = i32([0, 1])
    lens = i32([BS + tail] + [0] * forks)
    parents, children = i32([0] * forks), i32(range(1, forks + 1))
    free, count, left = i32(range(2, nb)), i32([forks]), i32([-1])
    status = i32([0])

    def fork():
        refs = i32([0] * nb)
        status.zero_()
        assert lib.paged_kv_fork(k.data_ptr(), v.data_ptr(), None, None, bt.data_ptr(), lens.data_ptr(),
                                 parents.data_ptr(), children.data_ptr(), refs.data_ptr(), free.data_ptr(),
                                 count.data_ptr(), left.data_ptr(), None, forks, forks + 1, H, D, 2, BS, forks, nb,
                                 torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        # fork i takes the block at the top of what is left of the stack
        assert bt[1:].cpu().tolist() == [[0, nb - 1 - i] for i in range(forks)]
        assert bool((lens == BS + tail).all()) and int(left) == 0 and int(refs[0]) == forks and int(refs.sum()) == forks
        copied = [bool((x[2:, :, :tail] == first[1, :, :tail]).all()) for x in (k, v)]
        rest = [bool((x[2:, :, tail:] == first[2:, :, tail:]).all()) for x in (k, v)]
        assert all(rest)
        return int(status), copied

    assert lib.paged_attn_set_checks(nb, status.data_ptr()) == 0
    lib.paged_attn_test_set_fork_fault((nb - 1) * H + 3)  # fork 0's rows of KV head 3
    got, copied = fork()
    assert got == 4 and copied == [False, False]
    # (a run goes in pieces of 4 KB, 16 rows of 256 bytes, and the first one is left out)
    assert bool((k[nb - 1, 3, :16] == first[nb - 1, 3, :16]).all())
    assert bool((k[2:nb - 20, :, :tail] == first[1, :, :tail]).all())  # other CTAs' runs
    lib.paged_attn_test_set_fork_fault(-1)
    assert fork() == (0, [True, True])


def test_rows_that_do_not_come_are_reported(lib):
    """8192 bf16 rows, streamed: the warp of the row that is missing ends, the others go on."""
    rows, H, D, BS = 8192, 8, 128, 16
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn(rows, H, D, generator=g, device="cuda").to(torch.bfloat16) for _ in "qkv")
    slots = torch.arange(rows, device="cuda")
    status = i32([0])

    def rope():
        out = torch.full_like(q, 7.0)
        kc, vc = (torch.full((rows // BS, H, BS, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        status.zero_()
        assert lib.paged_kv_rope_append_slots(q.data_ptr(), k.data_ptr(), v.data_ptr(), H * D, H * D, H * D,
                                              out.data_ptr(), kc.data_ptr(), vc.data_ptr(), None, None,
                                              slots.data_ptr(), None, 1, None, None, 1, 0, 0, None, None, 1e-6, rows,
                                              H, H, D, BS, rows // BS, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        dense = lambda c: c.transpose(1, 2).reshape(rows, H, D)
        same = [(a == b).flatten(1).all(1) for a, b in ((out, q), (dense(kc), k), (dense(vc), v))]
        return int(status), same

    assert lib.paged_attn_set_checks(rows // BS, status.data_ptr()) == 0
    lib.paged_attn_test_set_rope_fault(4000)
    got, same = rope()
    # (a warp has a few consecutive rows: 8192 of them over 16 warps an SM)
    assert got == 4 and not same[0][4000]
    assert all(bool(x[:3900].all()) and bool(x[4100:].all()) for x in same)
    lib.paged_attn_test_set_rope_fault(-1)
    got, same = rope()
    assert got == 0 and all(bool(x.all()) for x in same)
