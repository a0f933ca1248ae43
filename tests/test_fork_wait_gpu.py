"""The bounded waits of the forks' copies, made to run out on purpose: in a test build of the library
(``build.build_wait_test``, waits of a few milliseconds, never part of the product) two pages' first copies are
waited for and never issued.  The launch reports status bit 2, the warps that waited copy nothing more, and
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
    yield x
    x.paged_attn_test_set_fork_fault(-1)
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
