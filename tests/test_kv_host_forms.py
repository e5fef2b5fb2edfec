"""Sizes of the paged-cache calls for arguments without a bound, without a GPU."""
import ctypes

import pytest

import gguf_block_quantized_quantize_gb300 as g

FAR = 2 ** 63 - 1


def ws_size(**kw):
    a = dict(q=256, qt=g.BF16, n_tokens=20, ldq=512, cache=256, n_pages=4000, page_size=16, block_table=256, ld_table=4000,
             width=4000, q_start=256, kv_len=256, n_requests=1, max_q_len=20, n_heads=4, n_kv_heads=1, head_dim=128,
             scale=0.1, window=0, sinks=0, out=256, ldo=512, dev_status=0)
    a.update(kw)
    return g.load_library().gguf_paged_attention_ws_size(ctypes.byref(g.AttnArgs(*a.values())))


@pytest.mark.parametrize("far, near", [
    (dict(max_q_len=FAR), {}), (dict(window=FAR), {}), (dict(window=FAR, sinks=FAR), {}), (dict(window=2 ** 31), {}),
    (dict(window=9000, max_q_len=FAR), dict(window=9000)), (dict(window=9000, sinks=FAR), dict(window=9000, sinks=2 ** 31))])
def test_workspace_of_arguments_without_a_bound(far, near):
    """As for the bound that says the same: no request has more queries than the call, no position reaches 2^31."""
    assert ws_size(**far) == ws_size(**near) > 0
