"""GPU: paged attention where a key/value head has many query rows, and the calls that
share something: a broadcast query, a padded batch in a captured graph, one workspace for
two graphs. Tolerances as derived in test_attn_gpu.py."""
import math

import pytest
import torch

import gated_delta_rule_102_b200 as gdn
from attn_reference import attention
from test_attn_gpu import BF16, DEV, E4M3, F32, I32, Layer, check_attn, dev, view

pytestmark = pytest.mark.gpu

PAST = [0, 1, 47, 48, 63, 64, 65, 130, 777, 3000]


@pytest.mark.parametrize("d,G,T,ps", [
    (256, 3, 6, 8),        # 18 rows
    (256, 8, 16, 64),      # 128 rows, a whole tile
    (256, 16, 16, 48),     # two tiles
    (256, 11, 2, 16),      # 22 rows
    (128, 5, 16, 24),      # 80 rows: heads do not divide the tile
    (128, 12, 11, 64),     # 132 rows: four in the second tile
    (128, 15, 16, 128),    # 240 rows
    (128, 11, 3, 8),       # 33 rows
    (64, 6, 12, 1000),     # 72 rows
    (64, 13, 5, 40),       # 65 rows
    (64, 16, 16, 8),
    (256, 8, 16, 20),      # a page size that is no multiple of 8
    (64, 16, 16, 3),
])
def test_many_rows(d, G, T, ps):
    L = Layer(PAST, [T] * len(PAST), T, 2 * G, 2, d, ps, seed=d + G + T)
    check_attn(L, gated=G % 2 == 0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,softcap", [(1, 0.0), (5, 10.0), (64, 0.0), (100, 30.0), (0, 5.0)])
def test_many_rows_window_and_cap(d, window, softcap):
    L = Layer(PAST, [16] * len(PAST), 16, 16, 2, d, 32, seed=window, window=window, softcap=softcap)
    check_attn(L, window=window, softcap=softcap, gated=True)


def test_many_rows_ragged():
    counts = [0, 3, 16, 1, 0, 7, 2, 16, 0, 1, 1, 5, 0]
    L = Layer([50, 0, 1000, 2048, 9, 77, 300, 5, 0, 4095, 1, 640, 3], counts, 16, 16, 2, 256, 32, ragged=True)
    check_attn(L, gated=True)


@pytest.mark.parametrize("B,past", [(1, 30000), (150, 100), (2048, 2)])
def test_many_rows_splits(B, past):
    """One sequence over every CTA; several units in each; the largest batch."""
    L = Layer([max(0, past - 3 * (i % 20)) for i in range(B)], [5] * B, 5, 16, 1, 64 if B > 1000 else 128, 64)
    check_attn(L)


@pytest.mark.parametrize("d,window", [(256, 0), (128, 0), (64, 0), (256, 9), (128, 70)])
def test_many_rows_ignore_what_masks_leave_out(d, window):
    """NaN in pages of nobody, past the sequences and before the window; infinities in the
    last drafted token's value reach its own row alone."""
    T, past = 16, [0, 5, 15, 48, 100, 333]
    L = Layer(past, [T] * 6, T, 16, 2, d, 16, seed=d, window=window)
    kp, vp = L.pool(1.5), L.pool()
    keep = torch.zeros(L.pages, L.ps, dtype=torch.bool, device=DEV)
    for b, p in enumerate(past):
        pos = torch.arange(max(0, p + 1 - window) if window else 0, p + T)
        keep[L.table_cpu[L.slots_list[b]][pos // L.ps].to(DEV), (pos % L.ps).to(DEV)] = True
    for x in (kp, vp):
        x[~keep] = float("nan")
    for b, bad in ((2, float("inf")), (3, float("nan")), (5, float("-inf"))):
        pos = past[b] + T - 1
        vp[int(L.table_cpu[L.slots_list[b], pos // L.ps]), pos % L.ps, 0, ::3] = bad
    check_attn(L, window=window, k=kp, v=vp)


@pytest.mark.parametrize("d,G,T,kv", [(128, 4, 1, BF16), (128, 4, 1, E4M3), (64, 4, 4, BF16), (128, 4, 8, BF16), (256, 8, 2, BF16),
                                      (128, 16, 16, BF16), (256, 16, 4, BF16), (64, 8, 16, BF16)])
def test_attended_infinities(d, G, T, kv):
    """A key whose score is minus infinity has no weight, wherever it stands; a row whose
    scores hold a NaN is NaN, and only that row."""
    past = [0, 40, 64, 500]
    L = Layer(past, [T] * 4, T, G, 1, d, 16, kv, seed=d + T)
    ks, vs = (L.cfg.k_scale or 1.0, L.cfg.v_scale or 1.0)
    kp, vp, q = L.pool(1.5, ks), L.pool(1.0, vs), L.randn(4, T, G, d)
    q[..., 0] = q[..., 0].abs() + 0.5
    plain = kp.clone()
    where = []  # (sequence, position) of keys with a score of minus infinity
    if kv == BF16:
        where = [(1, i) for i in range(0, 33)] + [(2, i) for i in range(64)] + [(3, i) for i in range(500) if i % 64 < 40]
        for b, pos in where:
            page = int(L.table_cpu[L.slots_list[b], pos // 16])
            kp[page, pos % 16, 0, 0] = float("-inf")
            plain[page, pos % 16, 0] = 0
    out = torch.empty_like(q)
    lse = torch.empty(4, T, G, device=DEV)
    ws = gdn.attn_decode_workspace(L.cfg, 4, T, DEV)
    gdn.gdn_attn_decode(L.cfg, q, kp, vp, L.table, L.lens, L.slots, out, ws, lse=lse, err_flag=L.err)
    assert int(L.err) == 0
    for b in range(4):
        n = past[b] + T
        kk, vv = L.tokens(kp, b, n).double() * ks, L.tokens(vp, b, n).double() * vs
        want, wl, mass, _ = attention(q[b], kk, vv, past[b], 1 / math.sqrt(d), 0.0, 0)
        big = attention(q[b], L.tokens(plain, b, n).double() * ks, vv, past[b], 1 / math.sqrt(d), 0.0, 0)[3]
        eps_x = 2 * d * 2.0 ** -24 * big
        tol = (2 * eps_x + 2.0 ** -20 + (2.0 ** -8 if kv == BF16 else 2.0 ** -11))[..., None] * mass + 2.0 ** -8 * want.abs()
        assert torch.isfinite(want).all() and ((out[b].double() - want).abs() <= tol).all(), b
        assert ((lse[b].double() - wl).abs() <= eps_x + 2.0 ** -20 * (1 + wl.abs())).all()
    # a NaN in the last token's key: the rows before it do not attend it
    clean = out.clone()
    pos = past[3] + T - 1
    view(kp, kv)[int(L.table_cpu[L.slots_list[3], pos // 16]), pos % 16, 0, 1] = 0x7fc0 if kv == BF16 else 0x7f
    gdn.gdn_attn_decode(L.cfg, q, kp, vp, L.table, L.lens, L.slots, out, ws, lse=lse, err_flag=L.err)
    assert torch.isnan(out[3, -1]).all() and torch.isnan(lse[3, -1]).all()
    out[3, -1] = clean[3, -1]
    assert torch.equal(view(out, BF16), view(clean, BF16))


@pytest.mark.parametrize("d,G,T,kv", [(128, 4, 1, BF16), (256, 16, 4, BF16), (128, 8, 16, BF16), (64, 16, 16, E4M3)])
def test_broadcast_queries(d, G, T, kv):
    """One query row for all tokens, or one head for all heads (stride 0): as its copies."""
    L = Layer([30, 0, 700], [T] * 3, T, 2 * G, 2, d, 32, kv)
    kp, vp = L.pool(1.5, L.cfg.k_scale or 1.0), L.pool(1.0, L.cfg.v_scale or 1.0)
    ws = gdn.attn_decode_workspace(L.cfg, 3, T, DEV)

    def go(q):
        out = torch.empty(3, T, 2 * G, d, dtype=BF16, device=DEV)
        gdn.gdn_attn_decode(L.cfg, q, kp, vp, L.table, L.lens, L.slots, out, ws, err_flag=L.err)
        assert int(L.err) == 0
        return out

    one = L.randn(1, 1, 2 * G, d).expand(3, T, 2 * G, d)
    head = L.randn(3, T, 1, d).expand(3, T, 2 * G, d)
    both = L.randn(1, 1, 1, d).expand(3, T, 2 * G, d)
    for q in (one, head, both):
        check_attn(L, q=q, k=kp, v=vp)
        out, want = go(q), go(q.contiguous())
        # another kernel may serve the copies: both are within a rounding of the probabilities
        bound = 2.0 ** -7 + 2.0 ** -6 * vp.float().abs().max() * (L.cfg.v_scale or 1.0)
        assert ((out.float() - want.float()).abs() <= bound).all()


@pytest.mark.parametrize("Hq,d,kv", [(8, 128, BF16), (16, 256, BF16), (8, 128, E4M3)])
def test_padded_batch_in_a_graph(Hq, d, kv):
    """A captured step whose batch is padded: counts, slots and lengths change between
    replays, sequences of no tokens and rows past the last sequence stay as they were."""
    B, T, ps, Hkv = 6, 8, 16, 2
    L = Layer([0, 40, 100, 17, 300, 64], [T] * B, T, Hq, Hkv, d, ps, kv, rotary_dim=32)
    kp, vp = L.pool(1.5, L.cfg.k_scale or 1.0), L.pool(1.0, L.cfg.v_scale or 1.0)
    rows = B * T
    q, k, v = (L.randn(rows, h, d) for h in (Hq, Hkv, Hkv))
    inv = gdn.gdn_rope_inv_freq_host(32, 1e4)[0].to(DEV)
    cu = dev([0] * (B + 1))
    out, qo = torch.empty(rows, Hq, d, dtype=BF16, device=DEV), torch.empty(rows, Hq, d, dtype=BF16, device=DEV)
    ws = gdn.attn_decode_workspace(L.cfg, B, T, DEV)

    def step():
        gdn.gdn_qk_rope_append(L.cfg, q, k, v, None, None, inv, kp, vp, L.table, L.lens, L.slots, qo, cu_seqlens=cu, T_max=T, err_flag=L.err)
        gdn.gdn_attn_decode(L.cfg, qo, kp, vp, L.table, L.lens, L.slots, out, ws, cu_seqlens=cu, T_max=T, err_flag=L.err)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for counts in ([1, 0, 8, 3, 0, 0], [8] * 6, [0] * 6, [0, 0, 0, 0, 0, 5], [2, 1, 1, 1, 1, 8]):
        ends = torch.tensor([0] + counts).cumsum(0)
        cu.copy_(ends)
        out.fill_(-7.0)
        qo.fill_(-7.0)
        g.replay()
        assert int(L.err) == 0 and not ws[:576].any()
        used = int(ends[-1])
        assert (out[used:] == -7.0).all() and (qo[used:] == -7.0).all()
        ks, vs = (L.cfg.k_scale or 1.0, L.cfg.v_scale or 1.0)
        for b, n in enumerate(counts):
            if n == 0:
                continue
            r = slice(int(ends[b]), int(ends[b + 1]))
            kk, vv = L.tokens(kp, b, L.past[b] + n).double() * ks, L.tokens(vp, b, L.past[b] + n).double() * vs
            want, _, mass, big = attention(qo[r], kk, vv, L.past[b], 1 / math.sqrt(d), 0.0, 0)
            tol = (2.0 ** -8 + 2.0 ** -20 + 4 * d * 2.0 ** -24 * big)[..., None] * mass + 2.0 ** -8 * want.abs()
            assert ((out[r].double() - want).abs() <= tol).all(), (counts, b)


def test_two_graphs_share_a_workspace():
    """Graphs of different shapes (few rows, many rows), replayed in turn on one stream over
    one zeroed workspace that is large enough for both, beside eager calls."""
    A = Layer([900, 30, 0], [1] * 3, 1, 8, 2, 128, 16, seed=1)
    M = Layer([2000, 77], [16] * 2, 16, 16, 2, 128, 16, seed=2)
    size = max(gdn.attn_decode_workspace(L.cfg, L.B, L.T, DEV).numel() for L in (A, M))
    ws = torch.zeros(size, dtype=gdn.attn_decode_workspace(A.cfg, 1, 1, DEV).dtype, device=DEV)
    calls, graphs, want = [], [], []
    for L in (A, M):
        kp, vp, q = L.pool(1.5), L.pool(), L.randn(L.B, L.T, L.Hq, L.d)
        out = torch.empty_like(q)
        call = (L.cfg, q, kp, vp, L.table, L.lens, L.slots, out, ws)
        gdn.gdn_attn_decode(*call, err_flag=L.err)
        torch.cuda.synchronize()
        want.append(out.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gdn.gdn_attn_decode(*call, err_flag=L.err)
        calls.append(call)
        graphs.append(g)
    for i in range(20):
        for call in calls:
            call[7].zero_()
        for j in ((0, 1), (1, 0), (0, 0, 1, 1))[i % 3]:
            graphs[j].replay()
            gdn.gdn_attn_decode(*calls[1 - j])
        for call, w in zip(calls, want):
            assert torch.equal(view(call[7], BF16), view(w, BF16))
    assert int(A.err) == 0 and int(M.err) == 0 and not ws[:576].any()


def test_the_same_slot_twice_reads_the_same_cache():
    """Two rows of a batch may attend one sequence (the operator writes nothing of it)."""
    L = Layer([500, 20], [3, 3], 3, 16, 2, 128, 16)
    kp, vp = L.pool(), L.pool()
    slots = L.slots[[0, 1, 0]].contiguous()
    q = L.randn(3, 3, 16, 128)
    q[2] = q[0]
    out = torch.empty_like(q)
    gdn.gdn_attn_decode(L.cfg, q, kp, vp, L.table, L.lens, slots, out, gdn.attn_decode_workspace(L.cfg, 3, 3, DEV), err_flag=L.err)
    assert int(L.err) == 0
    # (their shares of the schedule differ, so the sums' order does)
    assert ((out[0].float() - out[2].float()).abs() <= 2.0 ** -6 * out[0].float().abs() + 2.0 ** -7).all()


@pytest.mark.parametrize("d,G,T", [(128, 4, 1), (128, 4, 4), (256, 8, 16), (64, 16, 16)])
@pytest.mark.parametrize("scale,softcap", [(-0.07, 0.0), (0.3, 0.0), (-0.2, 15.0)])
def test_score_factors_and_other_strides(d, G, T, scale, softcap):
    """A factor of its own, also a negative one; queries with heads outermost, one gate for all tokens."""
    L = Layer([0, 63, 500], [T] * 3, T, 2 * G, 2, d, 16, sm_scale=scale, softcap=softcap)
    kp, vp = L.pool(1.5), L.pool()
    q = L.randn(2 * G, 3, T, d).permute(1, 2, 0, 3)
    q = q.as_strided(q.shape, (T * d, d, 3 * T * d, 1))
    gate = L.randn(1, 1, 2 * G, d).expand(3, T, 2 * G, d)
    out = torch.empty(3, T, 2 * G, d, dtype=BF16, device=DEV)
    gdn.gdn_attn_decode(L.cfg, q, kp, vp, L.table, L.lens, L.slots, out, gdn.attn_decode_workspace(L.cfg, 3, T, DEV), gate=gate,
                        err_flag=L.err)
    assert int(L.err) == 0
    for b in range(3):
        n = L.past[b] + T
        kk, vv = L.tokens(kp, b, n), L.tokens(vp, b, n)
        want, _, mass, _ = attention(q[b], kk, vv, L.past[b], scale, softcap, 0, gate[b])
        big = attention(q[b], kk, vv, L.past[b], abs(scale), softcap, 0)[3]
        eps_x = 2 * d * 2.0 ** -24 * big + softcap * 2.0 ** -21
        tol = (2 * eps_x + 2.0 ** -20 + 2.0 ** -8)[..., None] * mass + 2.0 ** -8 * want.abs()
        assert ((out[b].double() - want).abs() <= tol).all(), b


@pytest.mark.parametrize("scale", [1e-30, 2.0 ** -80, 2.0 ** -40, 0.3, 1.0, 3.0, 1e25, 2.0 ** 100])
def test_append_divides_by_any_scale(scale):
    """Stored values are the quotients' roundings to the last bit, ties and the ends of the range among them."""
    d, Hkv, B = 128, 8, 64
    L = Layer([0] * B, [1] * B, 1, Hkv, Hkv, d, 1, E4M3)
    cfg = gdn.GdnAttnConfig.make(Hkv, Hkv, d, 1, kv_dtype=E4M3, k_scale=1.0, v_scale=scale)
    scale = cfg.v_scale  # (as 32 bits)
    q = L.randn(B, 1, Hkv, d)
    # quotients between e4m3's smallest and largest values, on and around its ties
    v = (torch.randn(B, 1, Hkv, d, generator=L.gpu, device=DEV).double() * 2.0 ** torch.randint(-11, 10, (B, 1, Hkv, d), generator=L.gpu, device=DEV)
         * scale).clamp(-3e38, 3e38).to(BF16)
    v[0, 0, 0, :6] = torch.tensor([0.0, -0.0, float("inf"), float("-inf"), 3e38, 1e-38]).to(BF16)
    kp, vp = L.pool(), L.pool()
    gdn.gdn_qk_rope_append(cfg, q, q, v, None, None, None, kp, vp, L.table, L.lens, L.slots, torch.empty_like(q), err_flag=L.err)
    assert int(L.err) == 0
    want = (v.float() / torch.full_like(v, scale, dtype=F32)).clamp(-448, 448).to(E4M3)
    page = L.table[L.slots.long(), 0].long()
    assert torch.equal(view(vp, E4M3)[page, 0], view(want, E4M3)[:, 0])
