"""GPU: attention over an e4m3 cache where one key outweighs a long tail that still counts.

A sink token of value zero stands above a flat tail, so the output is the tail's alone. Tolerances
as derived in test_attn_gpu.py: every probability that the fp16 products hold as a normal number
carries one rounding of 2^-11 of itself, however small it is next to the largest."""
import math

import pytest
import torch

import gated_delta_rule_102_b200 as gdn
from attn_reference import attention
from test_attn_gpu import BF16, DEV, E4M3, Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("above", [4, 12, 17, 18, 20])  # natural units; 20 is 2^-28.9
@pytest.mark.parametrize("d,G,T", [(256, 8, 8), (128, 8, 16), (64, 16, 16), (256, 8, 4), (128, 16, 1), (256, 8, 1), (64, 4, 2)])
def test_a_sink_above_a_flat_tail(d, G, T, above):
    past, B = 16000, torch.cuda.get_device_properties(0).multi_processor_count
    L = Layer([past], [T], T, G, 1, d, 64, E4M3, seed=above)
    cfg = gdn.GdnAttnConfig.make(G, 1, d, 64, kv_dtype=E4M3)
    # one element of the head makes the scores: `above` (as far as bf16 holds it) at the sink and 0 elsewhere
    kp = torch.zeros(L.pages, 64, 1, d, device=DEV).to(E4M3)
    vp = (L.randn(L.pages, 64, 1, d, std=0.5).float() + 1.0).to(E4M3)
    sink = int(L.table_cpu[L.slots_list[0], 0])
    kp.view(torch.uint8)[sink, 0, 0, 0] = 0x38  # 1.0
    vp.view(torch.uint8)[sink, 0] = 0
    q = torch.zeros(B, T, G, d, dtype=BF16, device=DEV)
    q[..., 0] = above * math.sqrt(d)
    # the sequence once for every SM: units stay whole, a piece of its own maximum would not tell
    slots = L.slots.expand(B).contiguous()
    out, lse = torch.empty_like(q), torch.empty(B, T, G, device=DEV)
    gdn.gdn_attn_decode(cfg, q, kp, vp, L.table, L.lens, slots, out, gdn.attn_decode_workspace(cfg, B, T, DEV), lse=lse,
                        err_flag=L.err)
    assert int(L.err) == 0
    kk, vv = L.tokens(kp, 0, past + T).double(), L.tokens(vp, 0, past + T).double()
    want, wl, mass, big = attention(q[0], kk, vv, past, 1 / math.sqrt(d), 0.0, 0)
    eps_x = 2 * d * 2.0 ** -24 * big
    tol = (2 * eps_x + 2.0 ** -20 + 2.0 ** -11)[..., None] * mass + 2.0 ** -8 * want.abs()
    off = ((out.double() - want).abs() / tol).amax()
    assert float(off) <= 1.0, float(off)
    assert ((lse.double() - wl).abs() <= eps_x + 2.0 ** -20 * (1 + wl.abs())).all()


@pytest.mark.parametrize("scale", [1e-36, 1e-30, 1e-3, 1e30])
@pytest.mark.parametrize("d,G,T,B", [(128, 4, 1, 3), (256, 8, 1, 148), (128, 8, 8, 148), (256, 8, 8, 3), (64, 16, 1, 3)])
def test_value_scales_of_every_size(scale, d, G, T, B):
    """The cache's scale is a factor of the output and of nothing else; 3000 tokens of about equal weight."""
    past = 3000
    L = Layer([past], [T], T, G, 1, d, 64, E4M3, seed=T)
    cfg = gdn.GdnAttnConfig.make(G, 1, d, 64, kv_dtype=E4M3, k_scale=0.0625, v_scale=scale)
    kp, vp, q = L.pool(1.5, 0.0625), L.pool(1.0, 0.03), L.randn(1, T, G, d, std=0.01).expand(B, T, G, d).contiguous()
    out = torch.empty_like(q)
    gdn.gdn_attn_decode(cfg, q, kp, vp, L.table, L.lens, L.slots.expand(B).contiguous(), out, gdn.attn_decode_workspace(cfg, B, T, DEV),
                        err_flag=L.err)
    assert int(L.err) == 0
    kk, vv = L.tokens(kp, 0, past + T).double() * 0.0625, L.tokens(vp, 0, past + T).double()
    want, _, mass, big = attention(q[0], kk, vv, past, 1 / math.sqrt(d), 0.0, 0)
    # in units of the scale; bf16's normal numbers end at 2^-126, a step below them is 2^-133
    eps_x = 2 * d * 2.0 ** -24 * big
    tol = (2 * eps_x + 2.0 ** -20 + 2.0 ** -11)[..., None] * mass + 2.0 ** -8 * want.abs() + 2.0 ** -133 / cfg.v_scale
    assert ((out.double() / cfg.v_scale - want).abs() <= tol).all()
