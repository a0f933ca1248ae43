"""The calls beside other streams, other threads and host memory: who may use the memory of an output that
a call makes, and when."""
import ctypes
import importlib.machinery
import importlib.util
import shutil
import subprocess
import threading
import time

import numpy as np
import pytest
import torch

import paged_kv_gqa_decode_gb300 as pa

pytestmark = pytest.mark.gpu

I32, BF = torch.int32, torch.bfloat16
SLEEP = 100_000_000  # cycles of a kernel that does nothing: about 50 ms


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_decode_gb300 import build

    build.build()
    pa.load()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=I32, device="cuda")


def normal(*shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(BF).cuda()


class Problem:
    """Two sequences of 40 and 23 tokens, the last 6 and 3 of them drafted, and a spare table row; 4 + 2 x 2
    heads of 128."""

    def __init__(self):
        self.k, self.v = normal(8, 2, 16, 128, seed=1), normal(8, 2, 16, 128, seed=2)
        self.q = normal(9, 4, 128, seed=3)
        self.kn, self.vn = normal(9, 2, 128, seed=4), normal(9, 2, 128, seed=5)
        self.bt = i32([[5, 1, 7], [0, 3, 6], [2, 4, 4]])
        self.lens, self.qo = i32([40, 23]), i32([0, 6, 9])
        self.mask = i32([[1], [3], [5], [11], [19], [33], [1], [3], [7]])
        self.slots = torch.arange(9, device="cuda") + 30
        self.pos = i32(list(range(9)))
        self.cs = torch.rand(16, 64, generator=torch.Generator().manual_seed(6)).cuda()
        self.free, self.count, self.refs = i32([2, 4, 0, 0, 0, 0, 0, 0]), i32([2]), i32([0] * 8)
        self.row_lens = i32([40, 23, 0])
        self.accepted, self.keep = i32([[0, 3, 5], [2, -1, -1]]), i32([17, 0])
        self.new = i32([3, 6])
        self.kx = self.k.view(8, 2, 16, 16, 8).transpose(2, 3).contiguous()
        self.parents, self.children = i32([0]), i32([2])
        self.ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")

    def tree(self, **kw):
        return [pa.paged_attn_decode_tree(self.q, self.k, self.v, self.qo, self.mask, self.bt[:2], self.lens, 0.1,
                                          workspace=self.ws, **kw)]

    def rope(self, **kw):
        return [pa.paged_kv_rope_append_slots(self.q, self.kn, self.vn, self.k, self.v, self.slots, self.pos,
                                              self.cs, **kw)]

    def compact(self, **kw):
        return [pa.paged_kv_compact(self.k, self.v, self.qo, self.accepted, self.bt[:2], self.lens, **kw)]

    def fork(self, **kw):
        return [pa.paged_kv_fork(self.k, self.v, self.bt, self.row_lens, self.parents, self.children, self.refs,
                                 self.free, self.count, **kw)]

    def release(self, **kw):
        return list(pa.paged_kv_release(self.bt[:2], self.lens, self.keep, self.free, self.count, 16, **kw))

    # those that are marshalled in Python
    def decode(self, **kw):
        return [pa.paged_attn_decode(self.q[:2], self.k, self.v, self.bt[:2], self.lens, 0.1, **kw)]

    def xpacked(self, **kw):
        return [pa.paged_attn_decode_xpacked(self.q[:2], self.kx, self.k.view(8, 2, 128, 16), self.bt[:2],
                                             self.lens, 0.1, **kw)]

    def multi(self, **kw):
        return [pa.paged_attn_decode_multi(self.q, self.k, self.v, self.qo, self.bt[:2], self.lens, 0.1, 6, **kw)]

    def append_decode(self, **kw):
        return [pa.paged_attn_append_decode(self.q[:2], self.kn[:2], self.vn[:2], self.k, self.v, self.bt[:2],
                                            self.lens, 0.1, **kw)]

    def mods(self, **kw):
        return [pa.paged_attn_decode_mods(self.q[:2], self.k, self.v, self.bt[:2], self.lens, 0.1, softcap=20.0,
                                          workspace=self.ws, **kw)]

    def multi_mods(self, **kw):
        return [pa.paged_attn_decode_multi_mods(self.q, self.k, self.v, self.qo, self.bt[:2], self.lens, 0.1,
                                                window=30, workspace=self.ws, **kw)]

    def assign(self, **kw):
        return list(pa.paged_kv_assign(self.lens, self.new, self.bt[:2], self.free, self.count, 16, 9, **kw))


CALLS = ["tree", "rope", "compact", "fork", "release"]
PYTHON = ["decode", "xpacked", "multi", "append_decode", "mods", "multi_mods", "assign"]


def crowd(sizes):
    """Live blocks, so that a freed one of these sizes is the one that the allocator gives next."""
    return [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(5000 if n < 512 else 200)]


@pytest.mark.parametrize("call", CALLS + PYTHON)
def test_made_outputs_are_the_given_streams_memory(call):
    """Blocks freed on the current stream with a write still to come do not become the outputs of a call on
    another stream."""
    want = getattr(Problem(), call)()
    s = torch.cuda.Stream()
    getattr(Problem(), call)(stream=s)  # (workspaces and kernels are there)
    p = Problem()
    sizes = [t.nbytes for t in want]
    held = crowd(sizes)
    torch.cuda.synchronize()
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda._sleep(SLEEP)
    for b in blocks:
        b.fill_(0x55)
    del b, blocks
    got = getattr(p, call)(stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    del held


@pytest.mark.parametrize("call", CALLS + PYTHON)
def test_a_dropped_output_is_not_given_to_the_current_stream_at_once(call):
    want = getattr(Problem(), call)()
    s = torch.cuda.Stream()
    getattr(Problem(), call)(stream=s)
    p = Problem()
    sizes = [t.nbytes for t in want]
    held = crowd(sizes)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SLEEP)
    getattr(p, call)(stream=s)  # runs after the sleep, into memory that nobody holds
    mine = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    assert all(bool((x == 0x55).all()) for x in mine)
    del held


@pytest.mark.parametrize("call", ["tree", "compact", "fork", "release", "assign", "mods", "multi_mods"])
def test_outputs_made_beside_pinned_inputs_are_device_memory(call):
    want = getattr(Problem(), call)()
    p = Problem()
    p.q, p.lens, p.count = (t.cpu().pin_memory() for t in (p.q, p.lens, p.count))
    got = getattr(p, call)()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert x.is_cuda and torch.equal(x, y)


# ------------------------------------------------------------------ other Python threads

@pytest.fixture
def slow(tmp_path, monkeypatch):
    """A second copy of the marshalling module whose entry points sleep on the host for 0.3 seconds, and then
    return the status that the fixture's function is given."""
    src, lib = tmp_path / "slow.c", tmp_path / "slow.so"
    src.write_text("#include <unistd.h>\nint status;\nint slow(void) { usleep(300000); return status; }\n")
    subprocess.run([shutil.which("gcc") or "gcc", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    stub = ctypes.CDLL(str(lib))
    path = shutil.copy(pa.NATIVE_PATH, tmp_path / "_paged_native.so")
    loader = importlib.machinery.ExtensionFileLoader("_paged_native", str(path))
    mod = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_paged_native", str(path),
                                                                                 loader=loader))
    loader.exec_module(mod)
    mod.init(pa._check, *[ctypes.cast(stub.slow, ctypes.c_void_p).value] * 5)
    monkeypatch.setattr(pa, "_native", mod)

    def returns(status):
        ctypes.c_int.in_dll(stub, "status").value = status

    return returns


@pytest.mark.parametrize("call", CALLS)
def test_other_threads_run_while_a_call_is_in_the_library(slow, call):
    p = Problem()
    torch.cuda.synchronize()
    ticks, done = [], threading.Event()

    def count():
        while not done.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.005)

    other = threading.Thread(target=count)
    other.start()
    try:
        start = time.perf_counter()
        getattr(p, call)()
        end = time.perf_counter()
        slow(-5)
        with pytest.raises(pa.PagedAttnError) as e:
            getattr(p, call)()
    finally:
        done.set()
        other.join()
    assert e.value.status == -5
    assert end - start > 0.2 and sum(start < t < end for t in ticks) >= 5


def test_calls_of_several_threads_at_once():
    """Each on a stream of its own, with outputs that the calls make."""
    want = {c: getattr(Problem(), c)() for c in CALLS}
    torch.cuda.synchronize()
    wrong = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(20):
            for c in CALLS:
                with torch.cuda.stream(s):
                    p = Problem()
                s.synchronize()
                got = getattr(p, c)(stream=s)
                s.synchronize()
                if not all(torch.equal(x, y) for x, y in zip(got, want[c])):
                    wrong.append(c)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []
