"""Numbers that the C ABI's types do not hold are refused by the binding: converted, a
window of 2^32 would be none, a cap below float32's range no cap.  No CUDA call is made."""
import pytest
import torch

import paged_kv_gqa_decode_gb300 as pa


def problem():
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    kc = torch.zeros(10, 2, 16, 128, dtype=torch.bfloat16)
    bt = torch.zeros(3, 4, dtype=torch.int32)
    return q, kc, kc.clone(), bt, torch.ones(3, dtype=torch.int32)


def calls(kw):
    q, kc, vc, bt, sl = problem()
    k8, f = torch.zeros(10, 2, 16, 128, dtype=torch.uint8), torch.zeros(10, 2, 16)
    qo = torch.arange(4, dtype=torch.int32)
    yield lambda: pa.paged_attn_decode_mods(q, kc, vc, bt, sl, 0.1, **kw)
    yield lambda: pa.paged_attn_decode_fp8_mods(q, k8, k8, f, f, bt, sl, 0.1, **kw)
    yield lambda: pa.paged_attn_decode_multi_mods(q, kc, vc, qo, bt, sl, 0.1, **kw)
    if "window" not in kw:
        yield lambda: pa.paged_attn_decode_shared(q, kc, vc, qo[:2], bt[:1], sl[:1], bt, sl, 0.1,
                                                  **kw)


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32, 2 ** 32 + 7, -2 ** 31 - 1])
def test_windows_past_32_bits(window):
    for call in calls(dict(window=window)):
        with pytest.raises(ValueError, match="window"):
            call()


@pytest.mark.parametrize("cap", [1e-50, -1e-60])
def test_caps_below_float32(cap):
    for call in calls(dict(softcap=cap)):
        with pytest.raises(ValueError, match="softcap"):
            call()


@pytest.mark.parametrize("kw,name", [(dict(block_size=2 ** 32 + 16, max_new=4), "block_size"),
                                     (dict(block_size=16, max_new=2 ** 32 + 4), "max_new")])
def test_sizes_of_an_assignment_past_32_bits(kw, name):
    x = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match=name):
        pa.paged_kv_assign(x, x, torch.zeros(2, 4, dtype=torch.int32), x, x[:1], **kw)
