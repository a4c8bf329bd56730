"""The attention layer's limits on sizes, from both sides, without a GPU: calls within a limit go on to
the check of alignment that follows it and are refused there (so nothing is enqueued on any machine)."""
import pytest
import torch

from test_attn_abi_cpu import FAKE, MIS, ODD2, ODD4, UNS, L, attn, cache, cfg, heads  # noqa: F401

LIMIT = 2 ** 31 - 2 ** 16


def ceil(a, b):
    return -(-a // b)


def places(Hkv, G, T, d, esz, positions, window, many):
    rows = T * G
    tile, row_tile = (64, 128 // G * G) if many else (8192 // (d * esz), next((r for r in (8, 16, 32, 64) if rows <= r), 64))
    positions = min(positions, window + T) if window else positions
    return Hkv * ceil(rows, row_tile) * (ceil(positions, tile) + 13)


@pytest.mark.parametrize("Hkv,G,T,d,kv,ps,window,many", [
    (8, 16, 16, 128, "bf16", 64, 0, True),
    (8, 9, 16, 128, "bf16", 64, 0, True),        # heads do not divide the row tile
    (8, 16, 16, 64, "bf16", 8, 0, True),
    (16, 16, 16, 256, "bf16", 20, 0, False),     # a page size for the other kernel
    (64, 8, 1, 256, "bf16", 64, 0, False),
    (64, 8, 2, 256, "e4m3", 64, 0, False),
    (128, 3, 8, 128, "e4m3", 16, 0, False),
    (512, 1, 1, 128, "bf16", 16, 0, False),
    (256, 4, 16, 256, "e4m3", 64, 100000, False),
    (256, 4, 16, 256, "bf16", 64, 300000, True),
])
def test_work_that_can_be_numbered(L, Hkv, G, T, d, kv, ps, window, many):
    """The largest batch or table within the limit, and the next one past it."""
    esz = 1 if kv == "e4m3" else 2
    c = cfg(num_q_heads=Hkv * G, num_kv_heads=Hkv, head_dim=d, page_size=ps, window=window, rotary_dim=0,
            kv_dtype=torch.float8_e4m3fn if kv == "e4m3" else torch.bfloat16)
    q = heads(row=Hkv * G * d, head=d)

    def call(B, pages):
        return attn(L, c, cache(max_pages=pages, num_pages=4), B=B, T=T, q=q, out=ODD4)

    pages = 0x7fff0000 // ps if window else ceil(262144, ps)
    one = places(Hkv, G, T, d, esz, pages * ps, window, many)
    B = LIMIT // one
    if B < 2048:
        assert call(B, pages) == MIS and call(B + 1, pages) == UNS
    if not window:  # and by the table's width, at the largest batch
        lo, hi = 1, 0x7fff0000 // ps
        while hi - lo > 1:
            mid = (lo + hi) // 2
            lo, hi = (mid, hi) if 2048 * places(Hkv, G, T, d, esz, mid * ps, 0, many) <= LIMIT else (lo, mid)
        assert call(2048, lo) == MIS and call(2048, lo + 1) == UNS


def test_short_sequences_in_wide_tables_are_served(L):
    """A table as wide as the longest context that a model takes, many drafted tokens, the largest batch."""
    c = cfg(num_q_heads=128, num_kv_heads=8, head_dim=128, page_size=64, rotary_dim=0)
    assert attn(L, c, cache(max_pages=131072 // 64), B=2048, T=16, q=heads(row=128 * 128, head=128), out=ODD4) == MIS
    assert attn(L, c, cache(max_pages=262144 // 64), B=1024, T=16, q=heads(row=128 * 128, head=128), out=ODD4) == MIS


def test_pools_and_tables_that_32_bits_can_walk(L):
    """Page numbers and table entries are walked in strides: within a stride of 2^31 an index would leave 32 bits."""
    F, most = FAKE, (1 << 31) - 1 - (1 << 15)
    calls = dict(reserve=lambda pages, width: L.gdn_pages_reserve(1, 2, F, F, 1, F, 4, width, F, F, pages, ODD2, None),
                 fork=lambda pages, width: L.gdn_pages_fork(1, 2, F, F, F, 4, width, F, F, pages, F, F, ODD2, None),
                 free=lambda pages, width: L.gdn_pages_free(2, F, F, 4, width, F, F, pages, ODD2, None),
                 compact=lambda pages, width: L.gdn_pages_compact(F, 4, width, F, pages, F, F, F, F, ODD2, None))
    for name, call in calls.items():
        assert call(most, 8) == MIS and call(8, most) == MIS, name
        assert call(most + 1, 8) == UNS and call((1 << 31) - 1, 8) == UNS, name
        assert call(8, most + 1) == UNS and call(8, (1 << 31) - 1) == UNS, name
