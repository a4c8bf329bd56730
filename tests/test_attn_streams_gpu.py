"""GPU: calls and plans of the attention layer run on the stream they are given, and on the current
one otherwise. What a call reads is written late on the stream that it should follow, and its output
holds a sentinel until then: a launch on any other stream reads the wrong values."""
import pytest
import torch

import gated_delta_rule_102_b200 as gdn
from test_attn_gpu import BF16, DEV, Layer, view

pytestmark = pytest.mark.gpu

LATE = 20_000_000  # cycles before the right values are written: ten milliseconds


@pytest.mark.parametrize("how", ["call, current", "call, given", "plan, current", "plan, given", "plan made for", "plan's, overridden", "elsewhere"])
@pytest.mark.parametrize("G,T", [(4, 1), (16, 8)])  # few and many rows
def test_order_on_a_stream(how, G, T):
    L = Layer([100, 2000], [T, T], T, 2 * G, 2, 128, 16, seed=G)
    kp, vp, right = L.pool(), L.pool(), L.randn(2, T, 2 * G, 128)
    want, out, q = (torch.empty_like(right) for _ in range(3))
    ws = gdn.attn_decode_workspace(L.cfg, 2, T, DEV)
    gdn.gdn_attn_decode(L.cfg, right, kp, vp, L.table, L.lens, L.slots, want, ws)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    plan = None
    args = (gdn.gdn_attn_decode, L.cfg, q, kp, vp, L.table, L.lens, L.slots, out, ws)
    if how.startswith("plan"):
        plan = gdn.CallPlan(*args, **({"stream": side} if how == "plan made for" else {"stream": other} if how == "plan's, overridden" else {}))
    for _ in range(2):
        q.zero_()
        out.fill_(-7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(LATE)
            q.copy_(right)
            if how == "call, current":
                gdn.gdn_attn_decode(*args[1:])
            elif how == "plan, current":
                plan.launch()
        if how == "call, given":
            gdn.gdn_attn_decode(*args[1:], stream=side)
        elif how == "plan made for":
            plan.launch()
        elif how in ("plan, given", "plan's, overridden"):
            plan.launch(stream=side)
        elif how == "elsewhere":  # what the other cases would see of a launch on a stream of its own
            gdn.gdn_attn_decode(*args[1:], stream=other)
        torch.cuda.synchronize()
        assert torch.equal(view(out, BF16), view(want, BF16)) == (how != "elsewhere")


def test_append_and_tables_on_a_stream():
    """The same of the append, the page tables and the copies, on a stream that is not the current one."""
    d, ps, side = 64, 16, torch.cuda.Stream()
    L = Layer([5], [1], 1, 2, 1, d, ps)
    x, right = torch.zeros(1, 1, 2, d, dtype=BF16, device=DEV), L.randn(1, 1, 2, d)
    kp, vp, out = L.pool(), L.pool(), torch.full((1, 1, 2, d), -7.0, dtype=BF16, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LATE)
        x.copy_(right)
    gdn.gdn_qk_rope_append(L.cfg, x, x[:, :, :1], x[:, :, 1:], None, None, None, kp, vp, L.table, L.lens, L.slots, out, stream=side)
    side.synchronize()
    page = int(L.table_cpu[L.slots_list[0], 0])
    assert torch.equal(out, right) and torch.equal(kp[page, 5], right[0, 0, :1]) and torch.equal(vp[page, 5], right[0, 0, 1:])

    table, lens = torch.full((3, 4), -1, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    refs, slots = torch.ones(6, dtype=torch.int32, device=DEV), torch.tensor([1], dtype=torch.int32, device=DEV)
    copy_src, copy_dst = (torch.full((1,), 9, dtype=torch.int32, device=DEV) for _ in range(2))
    data = torch.arange(6 * 8, dtype=torch.float32, device=DEV).view(6, 8)
    before, child = data.clone(), slots + 1
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LATE)
        refs[2:].zero_()  # until now no page is free
    gdn.gdn_pages_reserve(ps, slots, 20, table, lens, refs, stream=side)
    with torch.cuda.stream(side):
        lens[1] = 20
    gdn.gdn_pages_fork(ps, slots, child, table, lens, refs, copy_src, copy_dst, stream=side)
    gdn.gdn_copy_rows([data], copy_src, copy_dst, stream=side)
    side.synchronize()
    assert table.tolist() == [[-1] * 4, [2, 3, -1, -1], [2, 4, -1, -1]] and refs.tolist() == [1, 1, 2, 1, 1, 0]
    assert (copy_src.tolist(), copy_dst.tolist()) == ([3], [4])
    before[4] = before[3]
    assert torch.equal(data, before)
