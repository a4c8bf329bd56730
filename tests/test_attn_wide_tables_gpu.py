"""GPU: short sequences in tables that are as wide as a model's longest context, with the largest
batches. Tolerances as derived in test_attn_gpu.py."""
import math

import pytest
import torch

import gated_delta_rule_102_b200 as gdn
from attn_reference import attention
from test_attn_gpu import BF16, DEV, I32, Layer, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,positions,d", [(2048, 131072, 128), (1024, 262144, 64)])
def test_wide_tables(B, positions, d):
    T, G, Hkv, ps, past = 16, 16, 8, 64, [0, 63, 700, 5000]
    L = Layer(past, [T] * 4, T, G * Hkv, Hkv, d, ps, seed=d)
    table = torch.full((L.table.shape[0], positions // ps), -1, dtype=I32, device=DEV)
    table[:, :L.table.shape[1]] = L.table
    kp, vp = L.pool(1.5), L.pool()
    # the four sequences over and over; most without a token in this call, two with all
    counts = torch.zeros(B, dtype=torch.int64)
    counts[::7] = 1
    counts[[5, B - 1]] = T
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    total = int(cu[-1])
    slots = L.slots.repeat(B // 4)
    q = L.randn(total, G * Hkv, d, std=1.5)
    out, lse = torch.empty_like(q), torch.empty(total, G * Hkv, device=DEV)
    gdn.gdn_attn_decode(L.cfg, q, kp, vp, table, L.lens, slots, out, gdn.attn_decode_workspace(L.cfg, B, T, DEV), lse=lse,
                        cu_seqlens=dev(cu), T_max=T, err_flag=L.err)
    assert int(L.err) == 0 and q.dtype == BF16
    for b in [0, 5, 7, 14, 700, B - 1] + list(range(21, B, 203)):
        n, r = int(counts[b]), slice(int(cu[b]), int(cu[b + 1]))
        if n == 0:
            continue
        kk, vv = L.tokens(kp, b % 4, past[b % 4] + n), L.tokens(vp, b % 4, past[b % 4] + n)
        want, wl, mass, big = attention(q[r], kk, vv, past[b % 4], 1 / math.sqrt(d), 0.0, 0)
        eps_x = 2 * d * 2.0 ** -24 * big
        tol = (2 * eps_x + 2.0 ** -20 + 2.0 ** -8)[..., None] * mass + 2.0 ** -8 * want.abs()
        assert ((out[r].double() - want).abs() <= tol).all(), b
        assert ((lse[r].double() - wl).abs() <= eps_x + 2.0 ** -20 * (1 + wl.abs())).all(), b
