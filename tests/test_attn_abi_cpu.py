"""The softmax-attention layer's entry points on the host, without a GPU: every bad
argument is refused before anything is enqueued (fake pointers, never dereferenced), the
rotation speeds are checked against their formula, and the binding checks shapes."""
import ctypes
import math

import pytest
import torch

import gated_delta_rule_102_b200 as gdn
from gated_delta_rule_102_b200 import _attn
from gated_delta_rule_102_b200 import build as gdn_build

INV, UNS, MIS = gdn.GDN_ERR_INVALID_ARGUMENT, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_MISALIGNED
FAKE, ODD4, ODD2 = 1 << 20, (1 << 20) + 4, (1 << 20) + 2


@pytest.fixture(scope="module")
def L():
    gdn_build.build()
    return _attn._lib()


def cfg(**kw):
    base = dict(num_q_heads=16, num_kv_heads=2, head_dim=256, page_size=64, rotary_dim=64)
    base.update(kw)
    return gdn.GdnAttnConfig.make(**base)


def cache(**kw):
    base = dict(k_pages=FAKE, v_pages=FAKE, num_pages=10, page_table=FAKE, table_rows=4, max_pages=8, seq_lens=FAKE)
    base.update(kw)
    return _attn._KvCache(**base)


def heads(ptr=FAKE, row=4096, head=256):
    return _attn._Heads(ptr, row, head)


def append(L, c=None, kv=None, B=2, T=1, cu=None, total=None, q=None, k=None, v=None, qw=FAKE, kw=FAKE, inv=FAKE, slots=FAKE,
           out=FAKE, err=None):
    r = ctypes.byref
    return L.gdn_qk_rope_append(r(c or cfg()), r(kv or cache()), B, T, cu, B * T if total is None else total, r(q or heads()),
                                r(k or heads()), r(v or heads()), qw, kw, inv, slots, out, err, None)


def attn(L, c=None, kv=None, B=2, T=1, cu=None, total=None, q=None, gate=None, slots=FAKE, out=FAKE, lse=None, err=None, ws=FAKE):
    r = ctypes.byref
    return L.gdn_attn_decode(r(c or cfg()), r(kv or cache()), B, T, cu, B * T if total is None else total, r(q or heads()),
                             None if gate is None else r(gate), slots, out, lse, err, ws, None)


@pytest.mark.parametrize("call", [append, attn])
@pytest.mark.parametrize("kw,status", [
    (dict(num_q_heads=0), INV), (dict(num_kv_heads=-1), INV), (dict(num_q_heads=15), INV), (dict(head_dim=0), INV),
    (dict(page_size=0), INV), (dict(rotary_dim=63), INV), (dict(rotary_dim=258), INV), (dict(rotary_dim=-2), INV),
    (dict(window=-1), INV), (dict(norm_eps=-1.0), INV), (dict(norm_eps=float("nan")), INV), (dict(norm_offset=float("inf")), INV),
    (dict(sm_scale=float("nan")), INV), (dict(softcap=-1.0), INV), (dict(rope_scale=-1.0), INV), (dict(k_scale=2.0), INV),
    (dict(v_scale=0.5), INV), (dict(k_scale=float("inf"), kv_dtype=torch.float8_e4m3fn), INV),
    (dict(head_dim=96, rotary_dim=0), UNS), (dict(num_q_heads=34), UNS), (dict(page_size=65537), UNS),
])
def test_bad_configurations(L, call, kw, status):
    assert call(L, cfg(**kw)) == status


@pytest.mark.parametrize("call", [append, attn])
def test_bad_sizes_and_pointers(L, call):
    assert call(L, B=-1) == INV
    assert call(L, T=0) == INV
    assert call(L, T=17) == UNS
    assert call(L, B=2049) == UNS
    assert call(L, total=3) == INV                       # no offsets: B * T rows
    assert call(L, cu=ODD2, total=2) == MIS
    assert call(L, B=0) == gdn.GDN_OK and call(L, cu=FAKE, total=0) == gdn.GDN_OK
    for name in ("k_pages", "v_pages", "page_table", "seq_lens"):
        assert call(L, kv=cache(**{name: None})) == INV
    for name in ("k_pages", "v_pages"):
        assert call(L, kv=cache(**{name: ODD4})) == MIS
    for name in ("page_table", "seq_lens"):
        assert call(L, kv=cache(**{name: ODD2})) == MIS
    for name in ("num_pages", "table_rows", "max_pages"):
        assert call(L, kv=cache(**{name: 0})) == INV
    assert call(L, kv=cache(num_pages=1 << 30)) == UNS   # token numbers past 31 bits
    assert call(L, kv=cache(max_pages=1 << 26)) == UNS
    assert call(L, q=heads(None)) == INV
    assert call(L, q=heads(ODD4)) == MIS
    assert call(L, q=heads(row=-8)) == INV
    assert call(L, q=heads(row=4100)) == MIS
    assert call(L, q=heads(head=257)) == MIS
    assert call(L, slots=None) == INV and call(L, slots=ODD2) == MIS
    assert call(L, out=None) == INV and call(L, out=ODD4) == MIS
    assert call(L, err=ODD2) == MIS


def test_append_only(L):
    assert append(L, inv=None) == INV
    assert append(L, k=heads(None)) == INV and append(L, v=heads(head=4)) == MIS
    assert append(L, qw=ODD4) == MIS and append(L, kw=ODD4) == MIS and append(L, inv=ODD2) == MIS


def test_attn_only(L):
    assert attn(L, ws=None) == INV and attn(L, ws=ODD4) == MIS
    assert attn(L, lse=ODD2) == MIS
    assert attn(L, gate=heads(None)) == INV and attn(L, gate=heads(row=3)) == MIS
    big = cache(max_pages=(1 << 31) // 64 - 1)
    assert attn(L, kv=big, B=2048, T=16) == UNS          # too many token tiles to number
    assert gdn.attn_decode_workspace_bytes(cfg(), 4, 1) > 0
    assert gdn.attn_decode_workspace_bytes(cfg(head_dim=96, rotary_dim=0), 4, 1) == 0
    assert gdn.attn_decode_workspace_bytes(cfg(), 2049, 1) == 0 and gdn.attn_decode_workspace_bytes(cfg(), 1, 17) == 0


def test_page_entry_points(L):
    F = FAKE
    good = dict(reserve=[64, 2, F, F, 1, F, 4, 8, F, F, 10, None], fork=[64, 2, F, F, F, 4, 8, F, F, 10, F, F, None],
                free=[2, F, F, 4, 8, F, F, 10, None], compact=[F, 4, 8, F, 10, F, F, F, F, None])
    nullable = dict(reserve=(3,), fork=(), free=(), compact=())
    for name, args in good.items():
        f = getattr(L, "gdn_pages_" + name)
        for i, a in enumerate(args):
            if a == F:
                for bad, st in ((None, INV), (ODD2, MIS)):
                    if bad is None and i in nullable[name]:
                        continue
                    trial = list(args)
                    trial[i] = bad
                    assert f(*trial, None) == st, (name, i)
        trial = list(args)
        trial[-1] = ODD2
        assert f(*trial, None) == MIS
        sizes = dict(reserve=(0, 6, 7, 10), fork=(0, 5, 6, 9), free=(3, 4, 7), compact=(1, 2, 4))[name]
        for i in sizes:
            trial = list(args)
            trial[i] = 0
            assert f(*trial, None) == INV, (name, i)
        if name != "compact":
            n = 0 if name == "free" else 1
            trial = list(args)
            trial[n] = 2049
            assert f(*trial, None) == UNS
            trial[n] = -1
            assert f(*trial, None) == INV
            trial[n] = 0
            assert f(*trial, None) == gdn.GDN_OK
    assert L.gdn_pages_reserve(64, 2, F, None, -1, F, 4, 8, F, F, 10, None, None) == INV


def test_copy_rows(L):
    def copy(bufs, rows=4, n=2, src=FAKE, dst=FAKE, nd=None, err=None, count=None):
        a = (_attn._CopyBuffer * max(1, len(bufs)))(*[_attn._CopyBuffer(*b) for b in bufs])
        return L.gdn_copy_rows(a, len(bufs) if count is None else count, rows, n, src, dst, nd, err, None)
    ok = (FAKE, 64)
    assert copy([ok], n=0) == gdn.GDN_OK and copy([]) == gdn.GDN_OK
    assert copy([ok], rows=0) == INV and copy([ok], n=-1) == INV
    assert copy([ok], src=None) == INV and copy([ok], dst=ODD2) == MIS
    assert copy([ok], nd=ODD2) == MIS and copy([ok], err=ODD2) == MIS
    assert copy([(None, 64)]) == INV and copy([(FAKE, 0)]) == INV
    assert copy([ok, (ODD4, 64)]) == MIS and copy([(FAKE, 24)]) == MIS
    assert copy([ok] * 65) == UNS
    assert copy([(FAKE, 1 << 33)]) == UNS


def test_rotation_speeds(L):
    f, s = gdn.gdn_rope_inv_freq_host(64, 1e6)
    assert s == 1.0
    want = 1e6 ** (-torch.arange(32, dtype=torch.float64) / 32)
    assert torch.all((f.double() - want).abs() <= want * 2.0 ** -24)
    f4, s = gdn.gdn_rope_inv_freq_host(64, 1e6, factor=4.0)
    assert s == 1.0 and torch.all((f4.double() - want / 4).abs() <= want / 4 * 2.0 ** -24)
    y, s = gdn.gdn_rope_inv_freq_host(64, 1e6, factor=8.0, yarn=True, original_len=8192)
    assert abs(s - (0.1 * math.log(8.0) + 1)) < 1e-6
    turns = want * 8192 / (2 * math.pi)
    assert torch.equal(y[turns > 40], f[turns > 40])                    # fast pairs kept
    slow = y[turns < 0.7].double()
    assert torch.all((slow - want[turns < 0.7] / 8).abs() <= slow * 2.0 ** -23)
    assert torch.all(y[1:] < y[:-1]) and torch.all(y <= f) and torch.all(y.double() >= want / 8 * (1 - 2.0 ** -23))
    assert gdn.gdn_rope_inv_freq_host(0, 1e4)[0].numel() == 0
    for bad in ((63, 1e4, 1.0, False, 0), (64, 1.0, 1.0, False, 0), (64, 1e4, 0.5, False, 0), (64, 1e4, 2.0, True, 0),
                (-2, 1e4, 1.0, False, 0), (64, float("nan"), 1.0, False, 0)):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_rope_inv_freq_host(*bad)


def test_binding_refuses_cpu_tensors_and_foreign_functions():
    x = torch.zeros(1, 1, 16, 256, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    pages = torch.zeros(2, 64, 2, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        gdn.gdn_attn_decode(cfg(), x, pages, pages, i.view(2, 2), i[:2], i[:1], x, torch.zeros(1 << 24, dtype=torch.uint8))
    with pytest.raises(ValueError):
        gdn.gdn_attn_decode(cfg(), x, pages, pages, i.view(2, 2), i[:2], i[:1], x, torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        gdn.gdn_pages_free(i, i.view(2, 2), i[:2], i)
    with pytest.raises(TypeError):
        gdn.CallPlan(gdn.gdn_decode_step, 1)
    with pytest.raises(TypeError):
        gdn.GdnAttnConfig.make(16, 2, 256, 64, kv_dtype=torch.float16)


def test_positions_leave_room_for_a_tile(L):
    """A length near 2^31 would send a tile's end past it."""
    edge = (0x7fff0000 // 64)
    for call in (append, attn):
        assert call(L, kv=cache(max_pages=edge + 1)) == UNS
