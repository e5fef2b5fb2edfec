"""Forms of the paged-cache calls beyond the usual ones: one-sided norms, steps that hold more tokens than the
call, arguments without a bound, counts of what was left out, and queries whose values share a sign."""
import numpy as np
import pytest
import torch

import gguf_block_quantized_quantize_gb300 as g
from test_gpu_kv import DEV, DTYPES, HALF_ULP, attn_ref, attn_setup, check_attn, rope_ref

pytestmark = pytest.mark.gpu
I32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)   # noqa: E731


# ------------------------------------------------------------------ a norm of one side alone

@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("side", ["k", "q"])
@pytest.mark.parametrize("t, h, hk, d, neox", [
    (5, 0, 2, 128, True),        # keys alone
    (9, 4, 2, 64, False), (3, 6, 3, 256, True),
    (6000, 7, 3, 128, True),     # several rows per group of lanes, queries and keys among them
    (6000, 0, 9, 128, False)])
def test_norm_of_one_side(orc, typ, side, t, h, hk, d, neox):
    torch.manual_seed(t + h + d)
    dtype, eps, npos, page = DTYPES[typ], 1e-6, 500, 16
    q, k, v = (torch.randn(t, n, d, device=DEV).mul_(2).to(dtype) for n in (h, hk, hk))
    w = 1 + 0.2 * torch.randn(d, device=DEV)
    qw, kw = (w, None) if side == "q" else (None, w)
    ang = torch.rand(npos, d // 2, dtype=torch.float64) * 6.28
    table = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = torch.randint(0, npos, (t,), dtype=torch.int32)
    pages = -(-t // page) + 1
    slots = torch.randperm(pages * page)[:t].to(DEV)
    cache = torch.zeros(pages, g.gguf_kv_page_bytes(d, hk, page), dtype=torch.uint8, device=DEV)
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    g.gguf_qk_norm_rope(q, k, v, qw, kw, eps, pos.to(DEV), table.to(DEV), g.ROPE_NEOX if neox else g.ROPE_NORM,
                        cache=cache, slots=slots, page_size=page, q_out=q_out, k_out=k_out)
    cs = table.double()[pos.long()]
    gk, gv = g.gguf_kv_get_rows(cache, slots, hk, d, page)
    for got, x, xw in ((q_out, q, qw), (k_out, k, kw)):
        ref = rope_ref(x, xw, cs, d, neox, eps)
        # fp32: the norm's sum of d terms, four roundings, the rotation's three on terms up to |a| + |b|;
        # one rounding to the output type
        size = ref.abs() + ref.norm(dim=-1, keepdim=True) / np.sqrt(d) * 8
        assert bool(((got.double().cpu() - ref).abs() <= HALF_ULP[typ] * ref.abs() + 16 * 2.0 ** -24 * size).all())
    if typ == "f32":   # the stored blocks are Q4_0 of exactly the values that k_out shows
        held = orc.dequantize(orc.Q4_0, orc.quantize_weights(orc.Q4_0, k_out.reshape(-1, d).cpu().numpy()), d)
        assert torch.equal(gk.cpu(), torch.from_numpy(held.astype(np.float32)).view(gk.shape))
    else:              # within a code's step of the formula
        ref = rope_ref(k, kw, cs, d, neox, eps)
        step = (ref.unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True) / 8).expand(t, hk, d // 32, 32).flatten(-2)
        assert bool(((gk.double().cpu() - ref).abs() <= step * 1.01 + 1e-6).all())
