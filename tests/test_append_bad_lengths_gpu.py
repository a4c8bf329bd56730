"""GPU: sequences that an append skips for their lengths, among many that it does not: their CTAs leave
with rows of queries, keys and values on their way, the others' rows are those of a call without them."""
import pytest
import torch

import gated_delta_rule_102_b200 as gdn
from test_attn_gpu import BF16, DEV, E4M3, Layer, view

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,Hq,Hkv,kv", [(256, 16, 2, BF16), (128, 32, 8, E4M3), (64, 64, 8, BF16)])
def test_bad_lengths_among_many(d, Hq, Hkv, kv):
    B, T, ps = 512, 16, 16
    L = Layer([(7 * i) % 90 for i in range(B)], [T] * B, T, Hq, Hkv, d, ps, kv, seed=d, rotary_dim=d // 2)
    inv = gdn.gdn_rope_inv_freq_host(d // 2, 1e4)[0].to(DEV)
    q, k, v = (L.randn(B, T, h, d) for h in (Hq, Hkv, Hkv))
    kp, vp = L.pool(), L.pool()

    def go(lens, kp, vp, times):
        out = torch.full((B, T, Hq, d), -7.0, dtype=BF16, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        plan = gdn.CallPlan(gdn.gdn_qk_rope_append, L.cfg, q, k, v, None, None, inv, kp, vp, L.table, lens, L.slots, out, err_flag=err)
        for _ in range(times):
            plan.launch()
        return out, int(err)

    k1, v1, k2, v2 = kp.clone(), vp.clone(), kp.clone(), vp.clone()
    want, err = go(L.lens, k1, v1, 1)
    assert err == 0
    bad = torch.zeros(B, dtype=torch.bool, device=DEV)
    bad[::3] = True
    lens = L.lens.clone()
    slots = L.slots.long()
    lens[slots[bad]] = torch.where(torch.arange(int(bad.sum()), device=DEV) % 2 == 0, -1, L.table.shape[1] * ps - T + 1).int()
    out, err = go(lens, k2, v2, 20)
    assert err == gdn.GDN_DEVICE_ERR_SEQLEN
    assert (out[bad] == -7.0).all() and torch.equal(view(out[~bad], BF16), view(want[~bad], BF16))
    # the skipped sequences' places are as they were, the others' as without them
    for pool, full, before in ((k2, k1, kp), (v2, v1, vp)):
        expect = full.clone()
        for b in bad.nonzero().flatten().tolist():
            ids = L.table_cpu[L.slots_list[b]]
            ids = ids[ids >= 0].to(DEV)
            view(expect, kv)[ids] = view(before, kv)[ids]
        assert torch.equal(view(pool, kv), view(expect, kv))
