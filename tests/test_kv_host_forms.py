"""Sizes of the paged-cache calls for arguments without a bound, and the library beside its native module,
without a GPU."""
import ctypes
import os
import subprocess
import sys

import pytest

import gguf_block_quantized_quantize_gb300 as g

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

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


def test_products_without_the_native_module():
    """The module that marshals the paged-cache calls is theirs alone: the library loads and works without it."""
    code = ("import sys\n"
            "sys.modules['gguf_block_quantized_quantize_gb300._bind'] = None   # an import of it fails\n"
            "import gguf_block_quantized_quantize_gb300 as g\n"
            "assert g.gguf_row_size(g.Q4_0, 64) == 36 and g.gguf_get_option('mmq_enable') in (0, 1)\n"
            "assert g.gguf_kv_page_bytes(64, 1, 16) == 18 * 64\n"
            "try:\n"
            "    g._bound()\n"
            "except ImportError:\n"
            "    print('refused')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr
