"""GPU: the softmax-attention layer's operators against plain 64-bit restatements.

Tolerances. A rounding to bf16 is off by at most 2^-8 of the value, to fp16 2^-11, to
e4m3 2^-4 (half a step of the mantissa, or 2^-10 below the smallest normal).
append: the fp32 work before the rounding (a sum of d squares, a root, an angle rounded to
  32 bits after its reduction, four products) is off by less than 2e-6 of the rotated
  pair's magnitude.
attn: a score is a sum of d products in fp32, off by at most 2 d 2^-24 sum|q k| (twice the
  bound of a sum in any order); a probability carries that, the hardware exponential's
  2^-21 and, before it meets the values, one rounding (bf16 2^-8, fp16 2^-11). So
  |out - exact| <= (2 eps_x + 2^-20 + round_p) sum P|v| + 2^-8 |out|, and lse is off by at
  most eps_x + 2^-20 (1 + |lse|). A capped score adds c 2^-21 (the quotient in the tanh)."""
import math

import pytest
import torch

import gated_delta_rule_102_b200 as gdn
from attn_reference import attention, norm_rotate

pytestmark = pytest.mark.gpu
BF16, F32, I32, E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
DEV = "cuda"


def dev(x, dtype=I32):
    return torch.as_tensor(x, dtype=dtype).to(DEV)


class Layer:
    """A cache with its tables: sequences of given lengths in random slots and pages."""

    def __init__(self, past, counts, T, Hq, Hkv, d, ps, kv=BF16, seed=0, ragged=False, table_rows=None, **kw):
        self.cpu = torch.Generator().manual_seed(seed)
        self.gpu = torch.Generator(device=DEV).manual_seed(seed)
        self.past, self.counts, self.T, self.B = list(past), list(counts), T, len(past)
        rows = table_rows or self.B + 2
        self.slots_list = torch.randperm(rows, generator=self.cpu)[:self.B].tolist()
        held = [-(-(p + n) // ps) for p, n in zip(past, counts)]
        self.pages = sum(held) + 2
        ids = torch.randperm(self.pages, generator=self.cpu).tolist()
        table = torch.full((rows, max(held + [1])), -1, dtype=torch.int64)
        lens = torch.zeros(rows, dtype=torch.int64)
        at = 0
        for s, h, p in zip(self.slots_list, held, past):
            table[s, :h] = torch.tensor(ids[at:at + h], dtype=torch.int64)
            lens[s] = p
            at += h
        self.table_cpu = table
        self.table, self.lens, self.slots = dev(table), dev(lens), dev(self.slots_list)
        self.total = sum(counts)
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        self.cu_list, self.cu = cu, dev(cu) if ragged else None
        self.ps, self.Hq, self.Hkv, self.d, self.kv = ps, Hq, Hkv, d, kv
        scales = dict(k_scale=0.0625, v_scale=0.03) if kv == E4M3 else {}
        self.cfg = gdn.GdnAttnConfig.make(Hq, Hkv, d, ps, kv_dtype=kv, **scales, **kw)
        self.err = dev([0])

    def randn(self, *shape, std=1.0, dtype=BF16):
        return (torch.randn(*shape, generator=self.gpu, device=DEV) * std).to(dtype)

    def pool(self, std=1.0, scale=1.0):
        shape = (self.pages, self.ps, self.Hkv, self.d)
        if self.kv == BF16:
            return self.randn(*shape, std=std)
        return (torch.randn(*shape, generator=self.gpu, device=DEV) * (std / scale)).clamp(-448, 448).to(E4M3)

    def lead(self):
        return (self.total,) if self.cu is not None else (self.B, self.T)

    def tokens(self, pool, b, upto):
        ids = self.table_cpu[self.slots_list[b], :-(-upto // self.ps)].to(DEV)
        raw = pool.view(torch.uint8) if pool.dtype == E4M3 else pool
        return raw[ids].view(pool.dtype).flatten(0, 1)[:upto]


def view(x, dtype):
    return x.view(torch.int16 if dtype == BF16 else torch.uint8)


# ------------------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("d,R,inter,Hq,Hkv,ps,kv,T,ragged,gated", [
    (256, 64, False, 16, 2, 64, BF16, 1, False, True),
    (256, 256, True, 4, 4, 16, E4M3, 3, True, False),
    (128, 128, False, 32, 8, 24, BF16, 16, True, True),
    (128, 20, False, 5, 1, 1, E4M3, 2, False, False),     # halves of 10: partners across lanes
    (128, 6, True, 3, 3, 100, BF16, 1, False, False),
    (64, 64, False, 64, 8, 16, E4M3, 1, False, True),
    (64, 34, False, 8, 8, 8, BF16, 7, True, False),
    (64, 0, False, 1, 1, 32, BF16, 4, False, False),      # nothing rotated
    (256, 2, False, 70, 70, 5, BF16, 2, False, False),    # more heads than one batch of loads
])
def test_append(d, R, inter, Hq, Hkv, ps, kv, T, ragged, gated):
    past = [0, 5, 63, 64, 1000003 if Hkv * d <= 512 else 1900, 12345 if Hkv * d <= 512 else 17]  # (the pool holds them all)
    counts = [T, 0, 1, T, min(2, T), T] if ragged else [T] * 6
    L = Layer(past, counts, T, Hq, Hkv, d, ps, kv, seed=d + R, ragged=ragged, rotary_dim=R, rope_interleaved=inter,
              norm_offset=1.0, rope_scale=1.2 if inter else 0.0)
    inv, _ = gdn.gdn_rope_inv_freq_host(R, 1e6)
    qd = 2 * d if gated else d
    proj = L.randn(L.total, Hq * qd + 2 * Hkv * d)
    lead = L.lead()
    q = proj[:, :Hq * qd].view(*lead, Hq, qd)[..., :d]
    k = proj[:, Hq * qd:Hq * qd + Hkv * d].view(*lead, Hkv, d)
    v = proj[:, Hq * qd + Hkv * d:].view(*lead, Hkv, d)
    qw, kw = L.randn(d, std=0.1), L.randn(d, std=0.1)
    kp, vp = L.pool(), L.pool()
    k0, v0 = kp.clone(), vp.clone()
    out = torch.full(lead + (Hq, d), -7.0, dtype=BF16, device=DEV)
    gdn.gdn_qk_rope_append(L.cfg, q, k, v, qw, kw, inv.to(DEV) if R else None, kp, vp, L.table, L.lens, L.slots, out,
                           cu_seqlens=L.cu, T_max=T if ragged else None, err_flag=L.err)
    assert int(L.err) == 0
    pos = torch.cat([torch.arange(p, p + n) for p, n in zip(past, counts)]).to(DEV)
    b = torch.cat([torch.full((n,), i) for i, n in enumerate(counts)])
    rs = 1.2 if inter else 1.0
    flat = lambda x: x.reshape(L.total, x.shape[-2], d)  # noqa: E731
    y, mag = norm_rotate(flat(q), qw, 1.0, 1e-6, pos, inv, R, inter, rs)
    assert ((flat(out).double() - y).abs() <= 2.0 ** -8 * y.abs() + 2e-6 * mag).all()
    y, mag = norm_rotate(flat(k), kw, 1.0, 1e-6, pos, inv, R, inter, rs)
    page = L.table[L.slots[b.to(DEV)].long(), pos // ps].long()
    off = pos % ps
    ks, vs = (0.0625, 0.03) if kv == E4M3 else (1.0, 1.0)
    got = kp.to(F32)[page, off].double() * ks
    rel, low = (2.0 ** -8, 0.0) if kv == BF16 else (2.0 ** -4, 2.0 ** -10 * ks)
    assert ((got - y).abs() <= rel * y.abs() + low + 2e-6 * mag).all()
    if kv == BF16:
        assert torch.equal(vp[page, off], flat(v))
    else:
        # an element-wise division: torch divides by one number as a product with its rounded inverse
        want = (flat(v).float() / torch.full_like(flat(v), vs, dtype=F32)).clamp(-448, 448).to(E4M3)
        assert torch.equal(view(vp, kv)[page, off], view(want, kv))
    # every other place of the pools is as it was
    view(k0, kv)[page, off] = view(kp, kv)[page, off]
    view(v0, kv)[page, off] = view(vp, kv)[page, off]
    assert torch.equal(view(k0, kv), view(kp, kv)) and torch.equal(view(v0, kv), view(vp, kv))


def test_append_without_norms_and_saturating():
    d, Hq, Hkv = 128, 4, 2
    L = Layer([3, 40], [2, 2], 2, Hq, Hkv, d, 16, E4M3, rotary_dim=0)
    q, k, v = (L.randn(2, 2, h, d, std=100.0) for h in (Hq, Hkv, Hkv))
    k[0, 0, 0, :4] = dev([float("inf"), float("-inf"), float("nan"), 1e30], BF16)
    kp, vp = L.pool(), L.pool()
    out = torch.empty_like(q)
    gdn.gdn_qk_rope_append(L.cfg, q, k, v, None, None, None, kp, vp, L.table, L.lens, L.slots, out, err_flag=L.err)
    assert int(L.err) == 0 and torch.equal(out, q)
    s = L.slots_list[0]
    got = kp[int(L.table[s, 0]), 3, 0].float()
    want = (k[0, 0, 0].float() / 0.0625).clamp(-448, 448).to(E4M3).float()
    assert math.isnan(float(got[2])) and math.isnan(float(want[2]))
    assert torch.equal(got.nan_to_num(5.0), want.nan_to_num(5.0))


def test_append_skips_and_flags_bad_sequences():
    d, ps, B = 64, 16, 6
    L = Layer([0, 5, 17, 3, 16, 9], [2] * B, 2, 4, 2, d, ps, rotary_dim=64)
    inv = gdn.gdn_rope_inv_freq_host(64, 1e4)[0].to(DEV)
    q, k, v = (L.randn(B, 2, h, d) for h in (4, 2, 2))
    cases = []

    def bad(flag, rows, **kw):
        cases.append((flag, rows, kw))
    slots = L.slots.clone(); slots[1] = -1; slots[2] = 1000
    bad(gdn.GDN_DEVICE_ERR_SLOT_RANGE, [1, 2], slots=slots)
    lens = L.lens.clone(); lens[L.slots_list[0]] = -1; lens[L.slots_list[3]] = L.table.shape[1] * ps - 1
    bad(gdn.GDN_DEVICE_ERR_SEQLEN, [0, 3], lens=lens)
    table = L.table.clone(); table[L.slots_list[4], 1] = L.pages; table[L.slots_list[5], 0] = -1
    bad(gdn.GDN_DEVICE_ERR_PAGE, [], table=table)
    for flag, rows, kw in cases:
        kp, vp = L.pool(), L.pool()
        k0 = kp.clone()
        out = torch.full((B, 2, 4, d), -7.0, dtype=BF16, device=DEV)
        err = dev([0])
        gdn.gdn_qk_rope_append(L.cfg, q, k, v, None, None, inv, kp, vp, kw.get("table", L.table), kw.get("lens", L.lens),
                               kw.get("slots", L.slots), out, err_flag=err)
        assert int(err) == flag
        for b in range(B):
            assert bool((out[b] == -7.0).all()) == (b in rows)
        written = (kp != k0).flatten(2).any(-1).sum()
        assert int(written) == 2 * (B - len(rows)) - (4 if flag == gdn.GDN_DEVICE_ERR_PAGE else 0)


# -------------------------------------------------------------------------------------------------- attn
def check_attn(L, window=0, softcap=0.0, gated=False, k=None, v=None, q=None, launch=None, prepare=None):
    d, Hq, Hkv = L.d, L.Hq, L.Hkv
    ks, vs = (L.cfg.k_scale or 1.0, L.cfg.v_scale or 1.0)
    kp = L.pool(1.5, ks) if k is None else k
    vp = L.pool(1.0, vs) if v is None else v
    lead = L.lead()
    q = L.randn(*lead, Hq, d, std=1.5) if q is None else q
    gate = L.randn(*lead, Hq, 2 * d)[..., d:] if gated else None
    if prepare:
        prepare(L, kp, vp)
    out = torch.full(lead + (Hq, d), -7.0, dtype=BF16, device=DEV)
    lse = torch.full(lead + (Hq,), -7.0, device=DEV)
    ws = gdn.attn_decode_workspace(L.cfg, L.B, L.T, DEV)
    args = (L.cfg, q, kp, vp, L.table, L.lens, L.slots, out, ws)
    kw = dict(gate=gate, lse=lse, cu_seqlens=L.cu, T_max=L.T if L.cu is not None else None, err_flag=L.err)
    gdn.gdn_attn_decode(*args, **kw)
    first = out.clone(), lse.clone()
    gdn.gdn_attn_decode(*args, **kw)
    assert torch.equal(view(first[0], BF16), view(out, BF16)) and torch.equal(first[1].view(I32), lse.view(I32))
    assert int(L.err) == 0 and not ws[:576].any()
    scale = 1.0 / math.sqrt(d)
    worst = 0.0
    flat = lambda x: x.reshape(L.total, Hq, -1)  # noqa: E731
    o, ll = flat(out), lse.reshape(L.total, Hq)
    for b in range(L.B):
        n, r = L.counts[b], slice(L.cu_list[b], L.cu_list[b + 1])
        if n == 0:
            continue
        kk, vv = (L.tokens(x, b, L.past[b] + n).to(torch.float64) * s for x, s in ((kp, ks), (vp, vs)))
        want, wl, mass, big = attention(flat(q)[r], kk, vv, L.past[b], scale, softcap, window, None if gate is None else flat(gate)[r])
        eps_x = 2 * d * 2.0 ** -24 * big + softcap * 2.0 ** -21
        p = 2 * eps_x + 2.0 ** -20 + (2.0 ** -8 if L.kv == BF16 else 2.0 ** -11)
        tol = p[..., None] * mass + 2.0 ** -8 * want.abs()
        fine = torch.isfinite(want)
        assert torch.equal(torch.isfinite(o[r]), fine), f"sequence {b}"
        off = ((o[r].double() - want).abs() / (tol + 1e-30))[fine]
        assert off.numel() == 0 or float(off.max()) <= 1.0, (b, float(off.max()))
        le = ((ll[r].double() - wl).abs() / (eps_x + 2.0 ** -20 * (1 + wl.abs())))
        assert float(le.max()) <= 1.0, (b, float(le.max()))
        worst = max(worst, float(off.max()) if off.numel() else 0.0)
    return worst


LENGTHS = [0, 1, 14, 15, 16, 63, 64, 65, 127, 200, 511, 777]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kv", [BF16, E4M3])
@pytest.mark.parametrize("G,T", [(1, 1), (8, 1), (16, 1), (5, 3), (4, 8), (8, 16), (16, 16)])
def test_attn_heads_and_rows(d, kv, G, T):
    """One row tile of every height and several; every length around the tile edges."""
    L = Layer(LENGTHS, [T] * len(LENGTHS), T, 2 * G, 2, d, 16, kv, seed=G * T)
    check_attn(L, gated=T % 2 == 1)


@pytest.mark.parametrize("ps", [1, 7, 24, 64, 100, 1000])
@pytest.mark.parametrize("kv", [BF16, E4M3])
def test_attn_page_sizes(ps, kv):
    L = Layer([0, 99, 100, 101, 640, 1500], [2] * 6, 2, 8, 2, 128, ps, kv, seed=ps)
    check_attn(L)


@pytest.mark.parametrize("window,softcap", [(1, 0.0), (7, 20.0), (64, 0.0), (100, 50.0), (5000, 0.0), (0, 5.0)])
@pytest.mark.parametrize("d,kv,T", [(256, BF16, 1), (128, E4M3, 5), (64, BF16, 16), (256, E4M3, 16)])
def test_attn_window_and_cap(window, softcap, d, kv, T):
    L = Layer([0, 3, 64, 130, 700, 1300], [T] * 6, T, 8, 2, d, 16, kv, seed=window, window=window, softcap=softcap)
    check_attn(L, window=window, softcap=softcap, gated=True)


@pytest.mark.parametrize("kv", [BF16, E4M3])
def test_attn_ragged(kv):
    """Different counts, none among them; rows of no sequence are left as they were."""
    counts = [0, 3, 16, 1, 0, 7, 2, 16, 0, 1, 1, 5, 0]
    L = Layer([50, 0, 1000, 2048, 9, 77, 300, 5, 0, 4095, 1, 640, 3], counts, 16, 8, 1, 128, 32, kv, ragged=True)
    check_attn(L, gated=True)


@pytest.mark.parametrize("B,past,G,Hkv", [(1, 40000, 8, 2), (1, 0, 8, 2), (300, 70, 4, 2), (2048, 3, 1, 1), (3, 9000, 16, 8)])
def test_attn_splits(B, past, G, Hkv):
    """One long sequence over every CTA; many short ones in each CTA; more sequences than threads."""
    lens = [max(0, past - 3 * (i % 20)) for i in range(B)]
    L = Layer(lens, [1] * B, 1, G * Hkv, Hkv, 64 if B > 1000 else 128, 64)
    check_attn(L)


@pytest.mark.parametrize("d,kv,T,window", [(256, BF16, 1, 0), (128, E4M3, 4, 0), (128, BF16, 16, 20), (64, E4M3, 1, 9), (64, BF16, 3, 0)])
def test_attn_ignores_what_masks_leave_out(d, kv, T, window):
    """NaN and infinities past the sequences, in pages of nobody, before the window and in
    later drafted tokens reach no row that does not attend them."""
    past = [0, 5, 15, 16, 100, 333]
    L = Layer(past, [T] * 6, T, 4, 2, d, 16, kv, seed=T, window=window)

    def poison(L, kp, vp):
        for x, bad in ((kp, float("nan")), (vp, float("nan"))):
            keep = torch.zeros(L.pages, L.ps, dtype=torch.bool, device=DEV)
            for b, p in enumerate(past):
                ids = L.table_cpu[L.slots_list[b]]
                lo = max(0, p + 1 - window) if window else 0
                pos = torch.arange(lo, p + T)
                keep[ids[pos // L.ps].to(DEV), (pos % L.ps).to(DEV)] = True
            raw = view(x, L.kv)
            raw[~keep] = 0x7fc0 if L.kv == BF16 else 0x7f
        if T > 1:  # the last drafted token of two sequences: rows before it must stay finite
            for b in (3, 5):
                pos = past[b] + T - 1
                page = int(L.table_cpu[L.slots_list[b], pos // L.ps])
                view(vp, L.kv)[page, pos % L.ps, 0, ::3] = 0x7f80 if L.kv == BF16 else 0x7f
    if T > 1:
        # checked apart: the reference's own row for the poisoned token is not finite
        kp, vp = L.pool(1.5, L.cfg.k_scale or 1.0), L.pool(1.0, L.cfg.v_scale or 1.0)
        poison(L, kp, vp)
        check_attn(L, window=window, k=kp, v=vp)
    else:
        check_attn(L, window=window, prepare=poison)


def test_attn_extreme_scores():
    """Scores of thousands, one key that takes everything, equal keys, zero queries."""
    L = Layer([700, 64, 0, 1], [1] * 4, 1, 4, 1, 128, 16)
    q = L.randn(4, 1, 4, 128, std=60.0)
    q[1] = 0
    check_attn(L, q=q)
    L = Layer([700, 64, 0, 1], [1] * 4, 1, 4, 1, 128, 16, E4M3)
    q = L.randn(4, 1, 4, 128, std=3e4)
    q[1] = 0
    q[2, ..., ::2] *= 1e-6
    kp = (L.pool(1.0, 1.0).float() * 0.002).to(E4M3)
    check_attn(L, q=q, k=kp)


def test_attn_skips_and_flags_bad_sequences():
    B, ps, d = 6, 16, 128
    L = Layer([40, 5, 17, 3, 100, 9], [1] * B, 1, 4, 2, d, ps)
    q = L.randn(B, 1, 4, d)
    kp, vp = L.pool(), L.pool()
    ws = gdn.attn_decode_workspace(L.cfg, B, 1, DEV)

    def go(flag, rows, table=L.table, lens=L.lens, slots=L.slots, cu=None, unspecified=()):
        out = torch.full((B, 1, 4, d), -7.0, dtype=BF16, device=DEV)
        err = dev([0])
        gdn.gdn_attn_decode(L.cfg, q if cu is None else q.view(B, 4, d), kp, vp, table, lens, slots,
                            out if cu is None else out.view(B, 4, d), ws, cu_seqlens=cu, T_max=None if cu is None else 1, err_flag=err)
        assert int(err) == flag
        for b in range(B):
            if b not in unspecified:
                assert bool((out[b] == -7.0).all()) == (b in rows), b
        assert not ws[:576].any()
    go(0, [])
    slots = L.slots.clone(); slots[1] = -1; slots[2] = 1000
    go(gdn.GDN_DEVICE_ERR_SLOT_RANGE, [1, 2], slots=slots)
    lens = L.lens.clone(); lens[L.slots_list[0]] = -1; lens[L.slots_list[3]] = L.table.shape[1] * ps
    go(gdn.GDN_DEVICE_ERR_SEQLEN, [0, 3], lens=lens)
    table = L.table.clone(); table[L.slots_list[4], 3] = L.pages; table[L.slots_list[0], 0] = -1
    go(gdn.GDN_DEVICE_ERR_PAGE, [], table=table, unspecified=(0, 4))
    go(gdn.GDN_DEVICE_ERR_SEQLEN, [2, 3], cu=dev([0, 1, 2, 1, 4, 4 + 1, 6]), unspecified=(1,))
    go(0, [0, 5], cu=dev([1, 1, 2, 3, 4, 5, 5]))


def test_attn_far_offsets():
    """Pages past 2^32 bytes of the pool."""
    d, Hkv, ps = 256, 2, 256
    pages = (9 << 29) // (ps * Hkv * d * 2) + 3
    kp = torch.zeros(pages, ps, Hkv, d, dtype=BF16, device=DEV)
    L = Layer([300], [1], 1, 16, Hkv, d, ps)
    L.pages = pages
    L.table_cpu[L.slots_list[0], :2] = torch.tensor([pages - 1, pages - 3])
    L.table = dev(L.table_cpu)
    kp[-3:].copy_(L.randn(3, ps, Hkv, d))
    check_attn(L, k=kp, v=kp)
    inv = gdn.gdn_rope_inv_freq_host(0, 1e4)[0]
    k = L.randn(1, 1, Hkv, d)
    out = torch.empty(1, 1, 16, d, dtype=BF16, device=DEV)
    gdn.gdn_qk_rope_append(L.cfg, out, k, k, None, None, inv.to(DEV), kp, kp, L.table, L.lens, L.slots, out.clone(), err_flag=L.err)
    assert int(L.err) == 0 and torch.equal(kp[pages - 3, 300 - 256], k[0, 0])


# ----------------------------------------------------------------------- a run of the operators together
def test_layer_steps_in_a_graph():
    """Six decode steps of a layer (append, attend, lengths advanced on the device) as one
    captured graph, against the same steps made eagerly and against the reference; a second
    graph on a stream and workspace of its own runs at the same time."""
    B, T, Hq, Hkv, d, ps = 5, 2, 8, 2, 128, 16
    inv = gdn.gdn_rope_inv_freq_host(64, 1e4)[0]

    def make(seed):
        L = Layer([0, 13, 30, 64, 200], [T] * B, T, Hq, Hkv, d, ps, seed=seed, rotary_dim=64, norm_offset=1.0)
        width = (200 + 8 * T) // ps + 1
        table = torch.full((L.table.shape[0], width), -1)
        ids = iter(torch.randperm(B * width, generator=L.cpu).tolist())
        for s in L.slots_list:
            table[s] = torch.tensor([next(ids) for _ in range(width)])
        L.table_cpu, L.table, L.pages = table, dev(table), B * width
        return dict(L=L, kp=L.pool(), vp=L.pool(), x=L.randn(B, T, (Hq + 2 * Hkv) * d), qw=L.randn(d, std=0.1), kw=L.randn(d, std=0.1),
                    inv=inv.to(DEV), q=torch.empty(B, T, Hq, d, dtype=BF16, device=DEV), out=torch.empty(B, T, Hq, d, dtype=BF16, device=DEV),
                    ws=gdn.attn_decode_workspace(L.cfg, B, T, DEV))

    def step(s):
        L, x = s["L"], s["x"]
        q, k, v = (y.view(B, T, -1, d) for y in x.split([Hq * d, Hkv * d, Hkv * d], -1))
        gdn.gdn_qk_rope_append(L.cfg, q, k, v, s["qw"], s["kw"], s["inv"], s["kp"], s["vp"], L.table, L.lens, L.slots, s["q"], err_flag=L.err)
        gdn.gdn_attn_decode(L.cfg, s["q"], s["kp"], s["vp"], L.table, L.lens, L.slots, s["out"], s["ws"], err_flag=L.err)
        L.lens.index_add_(0, L.slots, torch.full((B,), T, dtype=I32, device=DEV))

    eager, a, b = make(1), make(1), make(2)
    b_eager = make(2)
    graphs = []
    for s in (a, b):
        lens0, kp0, vp0 = s["L"].lens.clone(), s["kp"].clone(), s["vp"].clone()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step(s)  # the first call sets up the host side
        stream.synchronize()
        s["L"].lens.copy_(lens0); s["kp"].copy_(kp0); s["vp"].copy_(vp0)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step(s)
        graphs.append((g, stream))
    torch.cuda.synchronize()
    for i in range(6):
        xs = [torch.randn(a["x"].shape, generator=a["L"].gpu, device=DEV).to(BF16) for _ in range(2)]
        torch.cuda.synchronize()
        for s, x, e, (g, stream) in zip((a, b), xs, (eager, b_eager), graphs):
            with torch.cuda.stream(stream):
                s["x"].copy_(x)
                g.replay()
            e["x"].copy_(x)
            step(e)
        torch.cuda.synchronize()
        for s, e in ((a, eager), (b, b_eager)):
            assert int(s["L"].err) == 0 and int(e["L"].err) == 0
            for key in ("out", "q", "kp", "vp"):
                assert torch.equal(view(s[key], BF16), view(e[key], BF16)), (i, key)
        L = eager["L"]
        for n in range(B):
            past = L.past[n] + i * T
            kk, vv = (L.tokens(x, n, past + T) for x in (eager["kp"], eager["vp"]))
            want, _, mass, big = attention(eager["q"][n], kk, vv, past, 1 / math.sqrt(d), 0.0, 0)
            tol = (2.0 ** -8 + 2.0 ** -20 + 4 * d * 2.0 ** -24 * big)[..., None] * mass + 2.0 ** -8 * want.abs()
            assert ((eager["out"][n].double() - want).abs() <= tol).all()


def test_plan_makes_the_same_call_and_another_stream_is_honoured():
    L = Layer([100, 2000], [1, 1], 1, 8, 2, 128, 16)
    kp, vp, q = L.pool(), L.pool(), L.randn(2, 1, 8, 128)
    out, again = torch.empty_like(q), torch.empty_like(q)
    ws = gdn.attn_decode_workspace(L.cfg, 2, 1, DEV)
    gdn.gdn_attn_decode(L.cfg, q, kp, vp, L.table, L.lens, L.slots, out, ws)
    torch.cuda.synchronize()
    plan = gdn.CallPlan(gdn.gdn_attn_decode, L.cfg, q, kp, vp, L.table, L.lens, L.slots, again, ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        q.neg_()  # the plan's launch must come after this, on the same stream
        q.neg_()
        plan.launch()
    side.synchronize()
    assert torch.equal(out, again)
    plan.launch(stream=side)
    side.synchronize()
    assert torch.equal(out, again)
