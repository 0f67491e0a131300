"""The calls on 8-bit caches, with positions of several axes and with shaped scores, on the CPU: the configuration is
checked before any device call, the binding refuses what the library cannot see, and what passes reaches the library in the
order the header declares, through the extension and without it."""
import ctypes
import os
import shutil
import subprocess
import threading
import time

import pytest

torch = pytest.importorskip("torch")

import hybrid_draft_tree_gb300 as g  # noqa: E402
from hybrid_draft_tree_gb300 import _build  # noqa: E402
from hybrid_draft_tree_gb300 import graft as gb  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E4M3 = torch.float8_e4m3fn


class FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


def kv_handle(eight=True, **over):
    cfg = g.graft_kv_default_config(4, 2, 64, 16, 8, 2, 4, g.GRAFT_BF16, cache="e4m3" if eight else None, **over)
    kv = object.__new__(g.GraftKV)
    kv.L, kv.cfg, kv.dtype, kv.h, kv.eight = FakeLib(), cfg, torch.bfloat16, None, eight
    kv.q_heads, kv.page_size, kv.rot_dim, kv.scale = cfg.q_heads, cfg.page_size, cfg.rot_dim, cfg.head_dim ** -0.5
    kv.q_width, kv.kv_width, kv.span = 256, 128, gb._cache_span(cfg)
    return kv


def bufs(kind=E4M3):
    bf, i32 = torch.bfloat16, lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(q=torch.zeros((8, 256), dtype=bf), k=torch.zeros((8, 128), dtype=bf), v=torch.zeros((8, 128), dtype=bf),
                rope=torch.zeros((32, 64)), table=i32(2, 2), ctx=i32(2), kc=torch.zeros((8, 2, 16, 64), dtype=kind),
                vc=torch.zeros((8, 2, 16, 64), dtype=kind), out=torch.zeros((8, 256), dtype=bf), pos=i32(2, 4), rows=i32(2, 4),
                pre=i32(2), mask=torch.zeros((2, 4), dtype=torch.int64), lse=torch.zeros((8, 4)), positions=i32(1, 2, 4),
                ks=torch.zeros(2), vs=torch.zeros(2), slopes=torch.zeros(4), first=i32(2), count=i32(2),
                ko=torch.zeros((8, 128), dtype=bf), vo=torch.zeros((8, 128), dtype=bf))


def calls(kv, b):
    return {
        "append": lambda: kv.append(2, 4, b["q"], b["k"], b["v"], b["rope"], b["table"], b["ctx"], b["kc"], b["vc"], b["out"],
                                    prefix_len=3, pos=b["pos"], rows=b["rows"], stream=0, positions=b["positions"],
                                    k_scale=b["ks"], v_scale=b["vs"]),
        "attend": lambda: kv.attend(2, 4, b["q"], b["kc"], b["vc"], b["table"], b["ctx"], 20, b["out"], prefix_pages=b["pre"],
                                    prefix_len=20, tree_mask=b["mask"], lse=b["lse"], stream=0, softcap=2.5, window=7,
                                    slopes=b["slopes"], k_scale=b["ks"], v_scale=b["vs"]),
        "read": lambda: kv.read(2, 4, b["kc"], b["vc"], b["table"], b["first"], b["count"], b["ko"], b["vo"], k_scale=b["ks"],
                                v_scale=b["vs"], stream=0),
    }


USED = {"append": ["q", "k", "v", "rope", "table", "ctx", "kc", "vc", "out", "pos", "rows", "positions", "ks", "vs"],
        "attend": ["q", "kc", "vc", "table", "ctx", "out", "pre", "mask", "lse", "slopes", "ks", "vs"],
        "read": ["kc", "vc", "table", "first", "count", "ko", "vo", "ks", "vs"]}


@pytest.fixture
def as_device(monkeypatch):
    monkeypatch.setattr(gb, "_on_device", lambda t: True)


def test_config_of_an_eight_bit_cache():
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    L = g.load()

    def init(dtype=g.GRAFT_BF16, dim=128, **over):
        cfg = g.graft_kv_default_config(8, 2, dim, 16, 10, 4, 61, dtype, **over)
        return L.graft_kv_init(ctypes.byref(cfg), ctypes.byref(ctypes.c_void_p()))

    for good in (dict(), dict(dtype=g.GRAFT_F16), dict(dim=64), dict(layout="token"), dict(page_stride=1 << 30),
                 dict(page_stride=4096 + 16)):
        assert init(cache="e4m3", **good) == gb.GRAFT_ECUDA, good
    for bad in (dict(page_stride=4096 + 8), dict(token_stride=136), dict(dtype=g.GRAFT_F32), dict(dtype=512 + 1),
                dict(head_stride=16 * 128 - 16)):
        assert init(cache="e4m3", **bad) == gb.GRAFT_EINVAL, bad
    assert init(page_stride=4096 + 8) == gb.GRAFT_ECUDA                       # of a 16-bit cache
    with pytest.raises(g.GraftError, match="cache"):
        g.graft_kv_default_config(8, 2, 128, 16, 10, 4, 61, cache="fp8")
    assert L.graft_kv_set_axes(None, 1, None) == gb.GRAFT_EINVAL
    for name, n in (("graft_kv_append_ext", 24), ("graft_kv_attend_ext", 21), ("graft_kv_read", 15)):
        args = [None if isinstance(t, type) and issubclass(t, (ctypes.c_void_p, ctypes._Pointer)) else t(0)
                for t in getattr(L, name).argtypes]
        assert len(args) == n and getattr(L, name)(*args) == gb.GRAFT_EINVAL  # a null handle


def test_structs_match_the_c_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    structs = {"graft_kv_scales": gb.graft_kv_scales, "graft_kv_scores": gb.graft_kv_scores}
    body = "".join(f'  printf("%zu\\n", sizeof({n}));\n' + "".join(f'  printf("%zu\\n", offsetof({n}, {f[0]}));\n' for f in c._fields_)
                   for n, c in structs.items())
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "graft.h"\nint main(void) {\n' + body +
                   '  printf("%d\\n", GRAFT_CACHE_E4M3);\n  return 0;\n}\n')
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "layout")])
    got = [int(x) for x in subprocess.check_output([str(tmp_path / "layout")]).split()]
    want = []
    for c in structs.values():
        want += [ctypes.sizeof(c)] + [getattr(c, f[0]).offset for f in c._fields_]
    assert got == want + [g.GRAFT_CACHE_E4M3]


@pytest.mark.parametrize("call", list(USED))
def test_host_buffers_are_refused(call):
    kv = kv_handle()
    with pytest.raises(g.GraftError, match="CUDA tensor") as e:
        calls(kv, bufs())[call]()
    assert e.value.code == gb.GRAFT_EINVAL and kv.L.calls == []


@pytest.mark.parametrize("kind", [E4M3, torch.uint8])
def test_valid_buffers_reach_the_library_in_abi_order(as_device, kind):
    kv, b = kv_handle(), bufs(kind)
    for f in calls(kv, b).values():
        f()
    p = {k: t.data_ptr() for k, t in b.items()}
    (n0, a0), (n1, a1), (n2, a2) = kv.L.calls
    assert n0 == "graft_kv_append_ext" and list(a0[:22]) == [
        None, 2, 4, p["q"], 256, p["k"], 128, p["v"], 128, p["pos"], p["rows"], p["positions"], p["rope"], 32, 3, p["table"], 2,
        p["ctx"], p["out"], 256, p["kc"], p["vc"]] and a0[23] == 0
    assert n1 == "graft_kv_attend_ext" and list(a1[:18]) == [
        None, 2, 4, p["q"], 256, p["kc"], p["vc"], p["pre"], 20, p["table"], 2, p["ctx"], 20, p["mask"], 0.125, p["out"], 256,
        p["lse"]] and a1[20] == 0
    assert n2 == "graft_kv_read" and list(a2[:9]) == [None, 2, 4, p["kc"], p["vc"], p["table"], 2, p["first"], p["count"]]
    assert list(a2[10:]) == [p["ko"], 128, p["vo"], 128, 0]
    for scales in (a0[22]._obj, a1[18]._obj, a2[9]._obj):
        assert (scales.d_k_scale, scales.d_v_scale) == (p["ks"], p["vs"])
    scores = a1[19]._obj
    assert (scores.softcap, scores.window, scores.d_slope) == (2.5, 7, p["slopes"])


@pytest.mark.parametrize("call,key", [(c, k) for c, keys in USED.items() for k in keys])
def test_each_buffer_is_checked(as_device, call, key):
    """Another element type, too few elements, a layout that is not the buffer's, no tensor at all."""
    good = bufs()[key]
    small = good[:-1] if good.dim() > 1 and good.shape[0] > 2 else good.flatten()[:-1]
    bad = [good.to(torch.float64), "text"]
    if key != "rope":                           # any number of positions
        bad.append(small)
    if key not in ("kc", "vc"):                 # reaches as far as the strides do
        bad.append(torch.zeros((*good.shape, 2), dtype=good.dtype)[..., 0])
    for x in bad:
        kv, b = kv_handle(), bufs()
        b[key] = x
        with pytest.raises(g.GraftError) as e:
            calls(kv, b)[call]()
        assert e.value.code == gb.GRAFT_EINVAL and kv.L.calls == [], x


def test_plain_calls_of_plain_handles_stay_what_they_are(as_device):
    """Without anything new a 16-bit handle makes the calls it made; with a 16-bit cache what is new but scales passes."""
    kv, b = kv_handle(eight=False), bufs(torch.bfloat16)
    args = (2, 4, b["q"], b["k"], b["v"], b["rope"], b["table"], b["ctx"], b["kc"], b["vc"], b["out"])
    kv.append(*args, stream=0)
    kv.attend(2, 4, b["q"], b["kc"], b["vc"], b["table"], b["ctx"], 20, b["out"], stream=0)
    kv.append(*args, stream=0, positions=b["positions"])
    kv.attend(2, 4, b["q"], b["kc"], b["vc"], b["table"], b["ctx"], 20, b["out"], stream=0, window=9)
    kv.read(2, 4, b["kc"], b["vc"], b["table"], b["first"], b["count"], b["ko"], b["vo"], stream=0)
    assert [n for n, _ in kv.L.calls] == ["graft_kv_append", "graft_kv_attend", "graft_kv_append_ext", "graft_kv_attend_ext",
                                          "graft_kv_read"]
    assert kv.L.calls[2][1][22] is None and kv.L.calls[3][1][18] is None and kv.L.calls[4][1][9] is None
    for f in calls(kv, b).values():
        with pytest.raises(g.GraftError, match="scales"):
            f()
    eight = kv_handle()
    with pytest.raises(g.GraftError, match="dtype"):
        eight.append(*args, stream=0)


def test_axes_are_checked(as_device):
    kv, b = kv_handle(), bufs()
    for bad in ([0] * 31, [0] * 33, []):
        with pytest.raises(g.GraftError, match="pairs"):
            kv.set_axes(bad)
    kv.set_axes([0, 1, 2, 0] * 8)
    name, (h, axes, pairs) = kv.L.calls.pop()
    assert name == "graft_kv_set_axes" and axes == 3 and list(pairs) == [0, 1, 2, 0] * 8 and kv.axes == 3
    with pytest.raises(g.GraftError, match="positions"):
        calls(kv, b)["append"]()                # one axis' positions
    b["positions"] = torch.zeros((3, 2, 4), dtype=torch.int32)
    calls(kv, b)["append"]()
    b["positions"] = torch.zeros((4, 2, 4), dtype=torch.int32)
    with pytest.raises(g.GraftError, match="positions"):
        calls(kv, b)["append"]()


class DeviceRows:
    """What the extension reads of a tensor, on a machine without a GPU."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.is_cuda = tuple(shape), dtype, True

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def stride(self):
        return tuple(DeviceRows(self.shape[i + 1:], self.dtype).numel() for i in range(len(self.shape)))


def extension():
    if _build.build_fastcall() is None:
        pytest.skip("no C compiler or Python headers")
    return gb._load_fastcall()


def fast_args(at, handle):
    bf, f32, i32, i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
    q, kv, cache = DeviceRows((8, 256), bf), DeviceRows((8, 128), bf), DeviceRows((8, 2, 16, 64), E4M3)
    table, ctx, rope, two = DeviceRows((2, 2), i32), DeviceRows((2,), i32), DeviceRows((32, 64), f32), DeviceRows((2,), f32)
    span = 8 * 2 * 16 * 64
    return {
        "append_ext": [at, handle, 0, bf, f32, i32, E4M3, 256, 128, 64, span, 2, 3, 2, 4, 0, q, kv, kv, rope, table, ctx, cache,
                       cache, q, None, None, DeviceRows((3, 2, 4), i32), two, None],
        "attend_ext": [at, handle, 0, bf, f32, i32, i64, E4M3, 256, 4, 16, span, 2, 2, 4, 0, 20, 5, 0.125, 2.0, q, cache, cache,
                       table, ctx, q, None, None, None, DeviceRows((4,), f32), two, two],
        "read": [at, handle, 0, bf, f32, i32, E4M3, 128, span, 2, 2, 4, cache, cache, table, ctx, ctx, kv, kv, two, two],
    }


def test_the_extension_frees_the_interpreter_lock_during_a_call():
    """usleep stands in for the library's entry points: the handle, its first argument, is how long it takes."""
    ext = extension()
    at = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    for name, args in fast_args(at, 300000).items():
        ticks, stop = [], threading.Event()

        def tick():
            while not stop.is_set():
                ticks.append(time.perf_counter())
                time.sleep(0.001)
        other = threading.Thread(target=tick)
        other.start()
        while not ticks:
            time.sleep(0.001)
        start = time.perf_counter()
        assert getattr(ext, name)(*args) == 0
        end = time.perf_counter()
        stop.set()
        other.join()
        assert end - start >= 0.2 and sum(start + 0.05 < t < end - 0.05 for t in ticks) >= 5, name


def test_the_extension_leaves_odd_arguments_to_the_binding():
    """Whatever is not as the checks want it is not called (the entry point's address would fault)."""
    ext = extension()
    wrong = [DeviceRows((1, 1), torch.float64), "text", 5]
    for name, good in fast_args(0, 0).items():
        first = {"append_ext": 16, "attend_ext": 20, "read": 12}[name]
        for i in range(first, len(good)):
            for x in wrong:
                args = list(good)
                args[i] = x
                assert getattr(ext, name)(*args) is NotImplemented, (name, i, x)
        assert getattr(ext, name)(*good[:-1]) is NotImplemented
    args = fast_args(0, 0)["append_ext"]
    args[27] = DeviceRows((4, 2, 4), torch.int32)      # another number of axes
    assert ext.append_ext(*args) is NotImplemented
    args = fast_args(0, 0)["attend_ext"]
    args[17] = 2 ** 31                                 # a window beyond 32 bits
    assert ext.attend_ext(*args) is NotImplemented
