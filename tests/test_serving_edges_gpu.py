"""Calls at the edges of what the serving entry points allow, on the GPU."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_decode_gb300 as pa
import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_decode_gb300 import build

    build.build()
    pa.load()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def test_no_groups_in_a_captured_stream():
    """A batch without shared prefixes: a workspace of the size that is asked for serves the
    captured call, whose output is the decode's."""
    w = workloads.make(workloads.custom_spec("none", 3, 8, 2, 128, 16, [5, 700, 33]), device="cuda")
    n = pa.paged_attn_shared_workspace_bytes(3, 0, 8, 2, 128, w.max_blocks_per_seq, 16)
    assert n >= pa.paged_attn_workspace_bytes(3, 8, 2, 128, w.max_blocks_per_seq, 16) > 0
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    none = (i32([0]), torch.zeros(0, 4, dtype=torch.int32, device="cuda"),
            torch.zeros(0, dtype=torch.int32, device="cuda"))
    out = torch.zeros_like(w.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.paged_attn_decode_shared(w.q, w.k_cache, w.v_cache, *none, w.block_tables, w.seq_lens,
                                    w.scale, out=out, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, pa.paged_attn_decode_mods(w.q, w.k_cache, w.v_cache, w.block_tables,
                                                      w.seq_lens, w.scale))
