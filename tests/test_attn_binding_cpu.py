"""The binding's numbers, without a GPU: what 32 bits do not hold is refused (ctypes would take its low
32 bits: a window of 2^32 + 5 would be one of 5)."""
import pytest

import gated_delta_rule_102_b200 as gdn
from gated_delta_rule_102_b200 import _attn
from test_attn_abi_cpu import L, cfg  # noqa: F401


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 16, 2 ** 63, -2 ** 31 - 1])
@pytest.mark.parametrize("field", ["num_q_heads", "num_kv_heads", "head_dim", "page_size", "rotary_dim", "window"])
def test_configurations(field, big):
    with pytest.raises(ValueError, match=field):
        cfg(**{field: big})


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 1, -2 ** 32 + 1])
def test_sizes(L, big):  # noqa: F811
    with pytest.raises(ValueError):
        gdn.attn_decode_workspace_bytes(cfg(), big, 1)
    with pytest.raises(ValueError):
        gdn.attn_decode_workspace_bytes(cfg(), 1, big)
    with pytest.raises(ValueError):
        gdn.gdn_rope_inv_freq_host(big, 1e4)
    with pytest.raises(ValueError):
        gdn.gdn_rope_inv_freq_host(64, 1e4, 2.0, True, big)
    none = (None,) * 12
    for at, name in ((0, "gdn_pages_reserve"), (4, "gdn_pages_reserve"), (2, "gdn_qk_rope_append"), (3, "gdn_attn_decode")):
        args = [0 if t is _attn.ctypes.c_int32 else x for t, x in zip(getattr(L, name).argtypes[:-1], none + none)]
        args[at] = big
        with pytest.raises(ValueError, match=name):
            _attn._Call(name, args, None, None)


def test_the_largest_numbers_pass(L):  # noqa: F811
    assert cfg(window=2 ** 31 - 1).window == 2 ** 31 - 1
    assert gdn.attn_decode_workspace_bytes(cfg(window=2 ** 31 - 1), 4, 1) == gdn.attn_decode_workspace_bytes(cfg(), 4, 1) > 0
