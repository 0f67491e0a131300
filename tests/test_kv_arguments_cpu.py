"""Numbers that the binding hands to the library in 32 bits: what 32 bits would make another call of is refused."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import hybrid_draft_tree_gb300 as g  # noqa: E402
from hybrid_draft_tree_gb300 import graft as gb  # noqa: E402
from test_kv_ext_cpu import bufs, extension, fast_args, kv_handle  # noqa: E402


@pytest.mark.parametrize("cap", [1e-50, 1e-46, -1e-50])
def test_a_cap_that_is_zero_in_32_bits_is_no_call_without_one(monkeypatch, cap):
    monkeypatch.setattr(gb, "_on_device", lambda t: True)
    kv, b = kv_handle(), bufs()
    with pytest.raises(g.GraftError, match="softcap") as e:
        kv.attend(2, 4, b["q"], b["kc"], b["vc"], b["table"], b["ctx"], 20, b["out"], stream=0, softcap=cap)
    assert e.value.code == gb.GRAFT_EINVAL and kv.L.calls == []
    args = fast_args(0, 0)["attend_ext"]
    args[19] = cap
    assert extension().attend_ext(*args) is NotImplemented      # left to the binding, which refuses it


def test_caps_that_are_numbers_in_32_bits_reach_the_library(monkeypatch):
    monkeypatch.setattr(gb, "_on_device", lambda t: True)
    for cap in (2.0 ** -149, 1e-30, 8e37):                      # the library judges how far they may be from the scale
        kv, b = kv_handle(), bufs()
        kv.attend(2, 4, b["q"], b["kc"], b["vc"], b["table"], b["ctx"], 20, b["out"], stream=0, softcap=cap)
        assert kv.L.calls[0][1][19]._obj.softcap == ctypes.c_float(cap).value
