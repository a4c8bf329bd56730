"""GPU: score caps of every size, from far below the scores to far above them, where a capped
score is all but the score itself.

Tolerances as derived in test_attn_gpu.py, with no part that grows with the cap: above 64 it is off by
at most 2^-20 of the score that it is given (and its slope is at most one), up to 64 by 1.2 c 2^-22, so a
score by eps_x = (2 d 2^-24 + 2^-20) sum|q k| + (1.2 c 2^-22 where c <= 64)."""
import math

import pytest
import torch

import gated_delta_rule_102_b200 as gdn
from attn_reference import attention
from test_attn_gpu import BF16, DEV, E4M3, Layer, view

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap", [1e-40, 1e-30, 1e-3, 0.7, 3.0, 30.0, 64.0, 65.0, 1e3, 1e4, 1e6, 1e9, 1e30, 3e38])
@pytest.mark.parametrize("d,kv,G,T", [(256, BF16, 8, 1), (128, E4M3, 4, 2), (128, BF16, 4, 3), (64, BF16, 8, 4), (256, E4M3, 8, 4),
                                      (256, BF16, 8, 16), (64, BF16, 16, 8)])
def test_caps_of_every_size(cap, d, kv, G, T):
    past = [0, 70, 900]
    L = Layer(past, [T] * 3, T, 2 * G, 2, d, 16, kv, seed=T, softcap=cap)
    ks, vs = (L.cfg.k_scale or 1.0, L.cfg.v_scale or 1.0)
    kp, vp, q = L.pool(1.5, ks), L.pool(1.0, vs), L.randn(3, T, 2 * G, d, std=1.5)
    q[1, 0, 0] = 0
    page = int(L.table_cpu[L.slots_list[2], 1])
    view(kp, kv)[page] = 0  # scores of zero whatever the query
    if cap < 1e-20:
        q[2] *= 4096
    out, lse = torch.empty_like(q), torch.empty(3, T, 2 * G, device=DEV)
    gdn.gdn_attn_decode(L.cfg, q, kp, vp, L.table, L.lens, L.slots, out, gdn.attn_decode_workspace(L.cfg, 3, T, DEV), lse=lse,
                        err_flag=L.err)
    assert int(L.err) == 0
    for b in range(3):
        n = past[b] + T
        kk, vv = L.tokens(kp, b, n).double() * ks, L.tokens(vp, b, n).double() * vs
        want, wl, mass, big = attention(q[b], kk, vv, past[b], 1 / math.sqrt(d), L.cfg.softcap, 0)
        eps_x = (2 * d * 2.0 ** -24 + 2.0 ** -20) * big + 1.2 * (cap if cap <= 64 else 0) * 2.0 ** -22
        tol = (2 * eps_x + 2.0 ** -20 + (2.0 ** -8 if kv == BF16 else 2.0 ** -11))[..., None] * mass + 2.0 ** -8 * want.abs()
        off = ((out[b].double() - want).abs() / tol).amax()
        assert float(off) <= 1.0, (b, float(off))
        le = ((lse[b].double() - wl).abs() / (eps_x + 2.0 ** -20 * (1 + wl.abs()))).amax()
        assert float(le) <= 1.0, (b, float(le))
