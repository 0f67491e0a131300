"""The paged-cache calls and the logit rules on the CPU: the handle's configuration is checked before any device call, the
binding's structs have the header's layout, its checks refuse what the library cannot see, and what passes reaches the
library in the order the header declares."""
import ctypes
import os
import shutil
import subprocess
import sysconfig
import threading
import time

import pytest

torch = pytest.importorskip("torch")

import hybrid_draft_tree_gb300 as g  # noqa: E402
from hybrid_draft_tree_gb300 import _build  # noqa: E402
from hybrid_draft_tree_gb300 import graft as gb  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


def kv_handle(**over):
    cfg = g.graft_kv_default_config(4, 2, 64, 16, 8, 2, 4, g.GRAFT_BF16, **over)
    kv = object.__new__(g.GraftKV)
    kv.L, kv.cfg, kv.dtype, kv.h = FakeLib(), cfg, torch.bfloat16, None
    kv.q_heads, kv.page_size, kv.rot_dim, kv.scale = cfg.q_heads, cfg.page_size, cfg.rot_dim, cfg.head_dim ** -0.5
    kv.q_width, kv.kv_width, kv.span = 256, 128, gb._cache_span(cfg)
    return kv


def graft_handle(V=100):
    eng = object.__new__(g.Graft)
    eng.L, eng.cfg, eng.S, eng.h = FakeLib(), g.graft_default_config(V, 2, g.GRAFT_MODE_STATIC, g.GRAFT_BF16), 61, None
    return eng


def bufs():
    bf, i32 = torch.bfloat16, lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(q=torch.zeros((8, 256), dtype=bf), k=torch.zeros((8, 128), dtype=bf), v=torch.zeros((8, 128), dtype=bf),
                rope=torch.zeros((32, 64)), table=i32(2, 2), ctx=i32(2), kc=torch.zeros((8, 2, 16, 64), dtype=bf),
                vc=torch.zeros((8, 2, 16, 64), dtype=bf), out=torch.zeros((8, 256), dtype=bf), pos=i32(2, 4),
                rows=i32(2, 4), pre=i32(2), mask=torch.zeros((2, 4), dtype=torch.int64), lse=torch.zeros((8, 4)),
                logits=torch.zeros((8, 100), dtype=bf), out_logits=torch.zeros((8, 100), dtype=bf), hist=i32(2, 9),
                hist_len=i32(2), prompt_len=i32(2), penalty=torch.zeros((2, 3)), bias_tok=i32(2, 5),
                bias_val=torch.zeros((2, 5)), grammar=i32(3, 4), grammar_row=i32(2, 4), tok=i32(2, 4))


def calls(kv, eng, b):
    return {
        "append": lambda: kv.append(2, 4, b["q"], b["k"], b["v"], b["rope"], b["table"], b["ctx"], b["kc"], b["vc"], b["out"],
                                    prefix_len=3, pos=b["pos"], rows=b["rows"], stream=0),
        "attend": lambda: kv.attend(2, 4, b["q"], b["kc"], b["vc"], b["table"], b["ctx"], 20, b["out"],
                                    prefix_pages=b["pre"], prefix_len=20, tree_mask=b["mask"], lse=b["lse"], stream=0),
        "logits": lambda: eng.process_logits(2, 4, b["logits"], b["out_logits"], tree_tok=b["tok"], tree_mask=b["mask"],
                                             hist=b["hist"], hist_len=b["hist_len"], prompt_len=b["prompt_len"],
                                             penalty=b["penalty"], bias_tok=b["bias_tok"], bias_val=b["bias_val"],
                                             grammar=b["grammar"], grammar_row=b["grammar_row"], stream=0),
    }


USED = {"append": ["q", "k", "v", "rope", "table", "ctx", "kc", "vc", "out", "pos", "rows"],
        "attend": ["q", "kc", "vc", "table", "ctx", "out", "pre", "mask", "lse"],
        "logits": ["logits", "out_logits", "tok", "mask", "hist", "hist_len", "prompt_len", "penalty", "bias_tok",
                   "bias_val", "grammar", "grammar_row"]}


@pytest.fixture
def as_device(monkeypatch):
    monkeypatch.setattr(gb, "_on_device", lambda t: True)


def test_config_is_checked_before_any_device_call():
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    L = g.load()

    def init(q=8, kv=2, dim=128, page=16, pages=10, batch=4, slots=61, dtype=g.GRAFT_BF16, **over):
        cfg = g.graft_kv_default_config(q, kv, dim, page, pages, batch, slots, dtype, **over)
        return L.graft_kv_init(ctypes.byref(cfg), ctypes.byref(ctypes.c_void_p()))

    for good in (dict(), dict(dim=64, dtype=g.GRAFT_F16), dict(layout="token"), dict(q=7, kv=7), dict(page=8),
                 dict(page=128, pages=(1 << 24) - 1), dict(rot_dim=0), dict(rot_dim=6, rot_interleaved=1),
                 dict(page_stride=1 << 30), dict(batch=1024, slots=63)):
        assert init(**good) == gb.GRAFT_ECUDA, good
    for bad in (dict(q=0), dict(kv=0), dict(q=7, kv=2), dict(q=2048, kv=2), dict(dim=96), dict(dim=256), dict(page=4),
                dict(page=24), dict(page=256), dict(pages=0), dict(page=128, pages=1 << 24), dict(batch=0), dict(slots=0),
                dict(slots=65), dict(batch=1100, slots=64), dict(dtype=g.GRAFT_F32), dict(rot_dim=-2), dict(rot_dim=3),
                dict(rot_dim=130), dict(rot_interleaved=2), dict(token_stride=120), dict(token_stride=132),
                dict(head_stride=16 * 128 - 8), dict(page_stride=2 * 16 * 128 - 8), dict(page_stride=1 << 38),
                dict(layout="token", head_stride=64)):
        assert init(**bad) == gb.GRAFT_EINVAL, bad
    with pytest.raises(g.GraftError, match="layout"):
        g.graft_kv_default_config(8, 2, 128, 16, 10, 4, 61, layout="page")
    with pytest.raises(g.GraftError):
        g.GraftKV(g.graft_kv_default_config(8, 2, 128, 16, 10, 4, 61))
    assert L.graft_kv_init(None, None) == gb.GRAFT_EINVAL
    for fn in (L.graft_kv_destroy, ):
        assert fn(None) == gb.GRAFT_EINVAL
    assert L.graft_kv_last_launch_count(None) == 0 and L.graft_kv_last_error(None) == b"null handle"


def test_strides_nest_in_any_order():
    """Tokens, heads and pages may lie in any order (heads outermost, as one buffer per head, among them); what overlaps is
    refused in each."""
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    L = g.load()

    def init(token, head, page, kv=2, ps=16, pages=10, dim=64):
        cfg = g.graft_kv_default_config(4, kv, dim, ps, pages, 2, 4, token_stride=token, head_stride=head, page_stride=page)
        return L.graft_kv_init(ctypes.byref(cfg), ctypes.byref(ctypes.c_void_p()))

    for token, head, page in ((64, 1024, 2048), (128, 64, 2048), (64, 10240, 1024), (640, 10240, 64), (1280, 64, 128),
                              (1280, 640, 64), (64, 10248, 1024), (72, 11520, 1152)):
        assert init(token, head, page) == gb.GRAFT_ECUDA, (token, head, page)
    for token, head, page in ((64, 10232, 1024), (64, 10240, 1016), (632, 10240, 64), (640, 10232, 64), (64, 64, 2048),
                              (1272, 64, 128), (1280, 632, 64), (1280, 64, 120), (64, 1024, 1024)):
        assert init(token, head, page) == gb.GRAFT_EINVAL, (token, head, page)
    assert init(64, 64, 1024, kv=1) == gb.GRAFT_ECUDA and init(64, 1024, 64, pages=1) == gb.GRAFT_ECUDA
    far = 1 << 37                                      # an extent beyond 64 bits
    assert init(far + 8, 64, far, ps=8, pages=(1 << 28) - 1, kv=1) == gb.GRAFT_EINVAL


def test_structs_match_the_c_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    structs = {"graft_kv_config": gb.graft_kv_config, "graft_logit_rules": gb.graft_logit_rules}
    body = "".join(f'  printf("%zu\\n", sizeof({n}));\n' + "".join(f'  printf("%zu\\n", offsetof({n}, {f[0]}));\n' for f in c._fields_)
                   for n, c in structs.items())
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "graft.h"\nint main(void) {\n' + body + "  return 0;\n}\n")
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "layout")])
    got = [int(x) for x in subprocess.check_output([str(tmp_path / "layout")]).split()]
    want = []
    for c in structs.values():
        want += [ctypes.sizeof(c)] + [getattr(c, f[0]).offset for f in c._fields_]
    assert got == want


@pytest.mark.parametrize("call", ["append", "attend", "logits"])
def test_host_buffers_are_refused(call):
    kv, eng = kv_handle(), graft_handle()
    with pytest.raises(g.GraftError, match="CUDA tensor") as e:
        calls(kv, eng, bufs())[call]()
    assert e.value.code == gb.GRAFT_EINVAL and kv.L.calls == [] and eng.L.calls == []


def test_valid_buffers_reach_the_library_in_abi_order(as_device):
    kv, eng, b = kv_handle(), graft_handle(), bufs()
    for f in calls(kv, eng, b).values():
        f()
    p = {k: t.data_ptr() for k, t in b.items()}
    (n0, a0), (n1, a1) = kv.L.calls
    assert n0 == "graft_kv_append" and list(a0) == [
        None, 2, 4, p["q"], 256, p["k"], 128, p["v"], 128, p["pos"], p["rows"], p["rope"], 32, 3, p["table"], 2, p["ctx"],
        p["out"], 256, p["kc"], p["vc"], 0]
    assert n1 == "graft_kv_attend" and list(a1) == [
        None, 2, 4, p["q"], 256, p["kc"], p["vc"], p["pre"], 20, p["table"], 2, p["ctx"], 20, p["mask"], 0.125, p["out"], 256,
        p["lse"], 0]
    (n2, a2), = eng.L.calls
    r = a2[7]._obj
    assert n2 == "graft_process_logits"
    assert list(a2[:7]) == [None, 2, 4, p["tok"], p["mask"], p["logits"], 100] and list(a2[8:]) == [p["out_logits"], 100, 0]
    assert (r.d_hist, r.hist_stride, r.d_hist_len, r.d_prompt_len, r.d_penalty) == (
        p["hist"], 9, p["hist_len"], p["prompt_len"], p["penalty"])
    assert (r.d_bias_tok, r.d_bias_val, r.n_bias, r.n_grammar, r.d_grammar, r.grammar_stride, r.d_grammar_row) == (
        p["bias_tok"], p["bias_val"], 5, 3, p["grammar"], 4, p["grammar_row"])


@pytest.mark.parametrize("call,key", [(c, k) for c, keys in USED.items() for k in keys])
def test_each_buffer_is_checked(as_device, call, key):
    """Another element type, too few elements, a layout that is not the buffer's, no tensor at all."""
    good = bufs()[key]
    wrong_type = good.to(torch.float64)
    small = good[:-1] if good.dim() > 1 and good.shape[0] > 2 else good.flatten()[:-1]
    strided = torch.zeros((*good.shape, 2), dtype=good.dtype)[..., 0]
    bad = [wrong_type, "text"]
    if key not in ("rope", "grammar"):          # any number of positions, of grammar rows
        bad.append(small)
    bad.append(strided)
    for x in bad:
        kv, eng, b = kv_handle(), graft_handle(), bufs()
        b[key] = x
        if key == "hist" and x is small:        # rows of another length are another history
            continue
        if key in ("kc", "vc") and x is strided:  # reaches as far as the strides do
            continue
        with pytest.raises(g.GraftError) as e:
            calls(kv, eng, b)[call]()
        assert e.value.code == gb.GRAFT_EINVAL and kv.L.calls == [] and eng.L.calls == [], x


def test_rows_keep_their_stride_and_options_are_null(as_device):
    kv, eng, b = kv_handle(), graft_handle(), bufs()
    qkv = torch.zeros((8, 512), dtype=torch.bfloat16)
    q, k, v = qkv.split([256, 128, 128], 1)
    kv.append(2, 4, q, k, v, b["rope"], b["table"], b["ctx"], b["kc"], b["vc"], b["out"], stream=0)
    kv.append(2, 4, None, k, v, b["rope"], b["table"], b["ctx"], b["kc"], b["vc"], None, stream=0)
    kv.attend(2, 4, q, b["kc"], b["vc"], b["table"], b["ctx"], 20, b["out"], stream=0, scale=1.5)
    (_, a0), (_, a1), (_, a2) = kv.L.calls
    assert list(a0[4:9:2]) == [512, 512, 512] and a0[9] is None and a0[10] is None
    assert a1[3] is None and a1[17] is None
    assert a2[7] is None and a2[13] is None and a2[14] == 1.5 and a2[17] is None
    wide = torch.zeros((8, 136), dtype=torch.bfloat16)[:, :100]
    eng.process_logits(2, 4, wide, b["out_logits"], stream=0)
    (_, a), = eng.L.calls
    assert a[6] == 136 and a[3] is None and a[7]._obj.d_hist is None and a[7]._obj.n_grammar == 0


def test_cache_reach_follows_the_strides(as_device):
    """A cache that is a slice of a larger buffer (one layer of interleaved pages) is held to the handle's strides."""
    layers = torch.zeros((8, 3, 2, 16, 64), dtype=torch.bfloat16)
    kv = kv_handle(page_stride=3 * 2 * 16 * 64)
    one = layers[:, 1]
    assert gb._cache(one, "k", torch.bfloat16, kv.span) == one.data_ptr()
    with pytest.raises(g.GraftError, match="elements"):
        gb._cache(layers[:7, 1], "k", torch.bfloat16, kv.span)


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


def test_the_extension_frees_the_interpreter_lock_during_a_call():
    """Other threads run while a call waits (for room in the launch queue, say).  usleep stands in for the library's entry
    points: the handle, its first argument, is how long it takes."""
    if _build.build_fastcall() is None:
        pytest.skip("no C compiler or Python headers")
    ext = gb._load_fastcall()
    at = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    bf, f32, i32, i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
    q, kv, cache = DeviceRows((8, 256), bf), DeviceRows((8, 128), bf), DeviceRows((8, 2, 16, 64), bf)
    table, ctx, rope = DeviceRows((2, 2), i32), DeviceRows((2,), i32), DeviceRows((32, 64), f32)
    x = DeviceRows((8, 100), bf)
    delay = 400000
    span = 8 * 2 * 16 * 64
    calls_ = {
        "append": (at, delay, 0, bf, f32, i32, 256, 128, 64, span, 2, 4, 0, q, kv, kv, rope, table, ctx, cache, cache, q, None, None),
        "attend": (at, delay, 0, bf, f32, i32, i64, 256, 4, 16, span, 2, 4, 0, 20, 0.125, q, cache, cache, table, ctx, q, None,
                   None, None),
        "logits": (at, delay, 0, bf, f32, i32, i64, 100, 2, 4, x, x, *[None] * 10),
    }
    for name, args in calls_.items():
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
        assert end - start >= 0.3, name
        assert sum(start + 0.05 < t < end - 0.05 for t in ticks) >= 5, name


def test_the_extension_is_named_for_its_interpreter():
    """An interpreter of another ABI looks for another file: it neither loads nor reuses this one's."""
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert sysconfig.get_config_var("SOABI") in suffix
    assert os.path.basename(_build.FASTCALL) == "_fastcall" + suffix


def test_accepted_rows_where_siblings_repeat_a_token():
    """The path is the verified one: the deepest, of equals the one that ends in the lowest slot, also when a lower slot
    with the same token has no child on it."""
    from workloads.target_model import accepted_rows
    tok = torch.tensor([[9, 4, 4, 5, 6, 6, -1], [9, 4, 5, 4, 5, 7, -1], [9, 1, 2, 3, -1, -1, -1], [9, 4, 4, 4, 5, 5, 8]],
                       dtype=torch.int32)
    parent = torch.tensor([[-1, 0, 0, 2, 3, 3, -1], [-1, 0, 1, 0, 3, 4, -1], [-1, 0, 0, 1, -1, -1, -1], [-1, 0, 0, 0, 3, 2, 1]],
                          dtype=torch.int8)
    emitted = torch.tensor([[4, 5, 6, 2, -1, -1, -1], [4, 5, 7, 1, -1, -1, -1], [5, -1, -1, -1, -1, -1, -1],
                            [4, 5, 0, -1, -1, -1, -1]], dtype=torch.int32)
    rows = accepted_rows(tok, parent, torch.tensor([3, 3, 0, 2], dtype=torch.int32), emitted)
    assert rows.tolist() == [[0, 2, 3, 4, -1, -1, -1], [0, 3, 4, 5, -1, -1, -1], [0, -1, -1, -1, -1, -1, -1],
                             [0, 3, 4, -1, -1, -1, -1]]
