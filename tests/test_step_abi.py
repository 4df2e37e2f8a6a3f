"""The C-ABI of include/df11_step.h: exported symbols, the binding's names and
what the host-side checks refuse.  No GPU work is started here; the pointers
handed in are never followed."""
import ctypes
import os
import re

import pytest

import huffman_decode_block_amd as hdb
from conftest import ROOT

P = 1 << 20  # an aligned address that only the host-side checks see


def declared_functions():
    src = open(os.path.join(ROOT, "include", "df11_step.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(df11_[a-z0-9_]+)\s*\(", src)))


def test_every_declared_symbol_is_exported_and_bound():
    names = declared_functions()
    lib = ctypes.CDLL(hdb.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
        assert callable(getattr(hdb, n)), n
        assert n in hdb.__all__, n
    assert sorted(hdb.STEP_EXPORTS) == names


@pytest.mark.parametrize("change", [
    dict(x=None), dict(x=P + 1), dict(codes=None), dict(codes=P + 8), dict(scales=None), dict(cols=0),
    dict(cols=(1 << 24) + 1, stride=(1 << 24) + 1), dict(stride=63), dict(rows=1 << 60), dict(rows=3, stride=1 << 62),
])
def test_quantise_refusals(change):
    a = dict(x=P, rows=2, cols=64, stride=64, codes=P, scales=P)
    a.update(change)
    L = hdb.lib()
    assert L.df11_mx4_quantize(a["x"], a["rows"], a["cols"], a["stride"], a["codes"], a["scales"], None) == \
        hdb.DF11_E_INVALID_ARG
    assert L.df11_mx4_dequantize(a["codes"], a["scales"], a["rows"], a["cols"], a["x"], a["stride"], None) == \
        hdb.DF11_E_INVALID_ARG


MANY = dict(m=4096, n=4096, ys=4096)  # rows and columns enough for the form that needs x readable or copied


@pytest.mark.parametrize("change,status", [
    (dict(x=None), hdb.DF11_E_INVALID_ARG), (dict(x=P + 1), hdb.DF11_E_INVALID_ARG),
    (dict(y=None), hdb.DF11_E_INVALID_ARG), (dict(y=P + 1), hdb.DF11_E_INVALID_ARG),
    (dict(codes=P + 4), hdb.DF11_E_INVALID_ARG), (dict(scales=None), hdb.DF11_E_INVALID_ARG),
    (dict(xs=63), hdb.DF11_E_INVALID_ARG), (dict(ys=39), hdb.DF11_E_INVALID_ARG),
    (dict(m=1 << 31), hdb.DF11_E_INVALID_ARG), (dict(n=1 << 31, ys=1 << 31), hdb.DF11_E_INVALID_ARG),
    (dict(k=(1 << 21) + 1, xs=1 << 25), hdb.DF11_E_INVALID_ARG), (dict(xs=1 << 33), hdb.DF11_E_INVALID_ARG),
    (dict(MANY, k=63), hdb.DF11_E_BUFFER_TOO_SMALL), (dict(MANY, x=P + 2), hdb.DF11_E_BUFFER_TOO_SMALL),
    (dict(MANY, xs=65), hdb.DF11_E_BUFFER_TOO_SMALL), (dict(MANY, k=63, ws=P + 8, size=1 << 30), hdb.DF11_E_INVALID_ARG),
    (dict(MANY, k=63, ws=None, size=1 << 30), hdb.DF11_E_INVALID_ARG),
])
def test_product_refusals(change, status):
    a = dict(x=P, m=3, k=64, xs=64, codes=P, scales=P, n=40, y=P, ys=40, ws=None, size=0)
    a.update(change)
    got = hdb.lib().df11_mx4_matmul(a["x"], a["m"], a["k"], a["xs"], a["codes"], a["scales"], a["n"], a["y"], a["ys"],
                                    a["ws"], a["size"], None)
    assert got == status


def test_empty_calls_need_no_pointers():
    L = hdb.lib()
    assert L.df11_mx4_quantize(None, 0, 64, 64, None, None, None) == hdb.DF11_OK
    assert L.df11_mx4_dequantize(None, None, 0, 64, None, 64, None) == hdb.DF11_OK
    assert L.df11_mx4_matmul(None, 0, 64, 64, None, None, 40, None, 40, None, 0, None) == hdb.DF11_OK
    assert L.df11_mx4_matmul(None, 3, 64, 64, None, None, 0, None, 0, None, 0, None) == hdb.DF11_OK
    c = cache()
    assert L.df11_paged_append(ctypes.byref(c), None, 0, 0, None, 0, 0, None, 0, None) == hdb.DF11_OK
    assert L.df11_paged_attention(ctypes.byref(c), None, 0, 8, 0, 0, None, 4, 4, None, None, 1.0, None, None, None, 0,
                                  None) == hdb.DF11_OK


def cache(**change):
    a = dict(k_pages=P, v_pages=P, n_pages=10, k_page_stride=16384, k_head_stride=2048, k_row_stride=128,
             v_page_stride=16384, v_head_stride=2048, v_row_stride=128, k_scale=None, v_scale=None, kv_heads=8,
             head_dim=128, page_size=16, dtype=hdb.DF11_CACHE_BF16)
    a.update(change)
    return hdb.step.df11_paged_cache(**a)


BAD_CACHES = [
    (dict(k_pages=None), hdb.DF11_E_INVALID_ARG), (dict(v_pages=P + 2), hdb.DF11_E_INVALID_ARG),
    (dict(n_pages=0), hdb.DF11_E_INVALID_ARG), (dict(n_pages=1 << 31), hdb.DF11_E_INVALID_ARG),
    (dict(kv_heads=0), hdb.DF11_E_INVALID_ARG), (dict(k_row_stride=129), hdb.DF11_E_INVALID_ARG),
    (dict(v_head_stride=1 << 41), hdb.DF11_E_INVALID_ARG), (dict(head_dim=96), hdb.DF11_E_UNSUPPORTED),
    (dict(head_dim=0), hdb.DF11_E_UNSUPPORTED), (dict(page_size=4), hdb.DF11_E_UNSUPPORTED),
    (dict(page_size=24), hdb.DF11_E_UNSUPPORTED), (dict(page_size=2048), hdb.DF11_E_UNSUPPORTED),
    (dict(dtype=2), hdb.DF11_E_UNSUPPORTED), (dict(dtype=hdb.DF11_CACHE_E4M3), hdb.DF11_E_INVALID_ARG),
    (dict(dtype=hdb.DF11_CACHE_E4M3, k_scale=P, v_scale=P, k_row_stride=136), hdb.DF11_E_INVALID_ARG),
]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_cache_refusals(change, status):
    L = hdb.lib()
    c = ctypes.byref(cache(**change))
    assert L.df11_paged_append(c, P, 1024, 128, P, 1024, 128, P, 1, None) == status
    assert L.df11_paged_attention(c, P, 1, 8, 1024, 128, P, 4, 4, P, None, 1.0, P, P, None, 0, None) == status


@pytest.mark.parametrize("change", [dict(k=None), dict(v=P + 1), dict(slots=None), dict(slots=P + 4), dict(tokens=1 << 31),
                                    dict(stride=1 << 41)])
def test_append_refusals(change):
    a = dict(k=P, v=P, slots=P, tokens=2, stride=1024)
    a.update(change)
    c = cache()
    assert hdb.lib().df11_paged_append(ctypes.byref(c), a["k"], a["stride"], 128, a["v"], a["stride"], 128, a["slots"],
                                       a["tokens"], None) == hdb.DF11_E_INVALID_ARG
    assert hdb.lib().df11_paged_append(None, P, 0, 0, P, 0, 0, P, 1, None) == hdb.DF11_E_INVALID_ARG


@pytest.mark.parametrize("change,status", [
    (dict(q=None), hdb.DF11_E_INVALID_ARG), (dict(out=None), hdb.DF11_E_INVALID_ARG), (dict(table=None), hdb.DF11_E_INVALID_ARG),
    (dict(lens=None), hdb.DF11_E_INVALID_ARG), (dict(lens=P + 2), hdb.DF11_E_INVALID_ARG), (dict(starts=P + 1), hdb.DF11_E_INVALID_ARG),
    (dict(lse=P + 2), hdb.DF11_E_INVALID_ARG), (dict(heads=12), hdb.DF11_E_INVALID_ARG), (dict(heads=0), hdb.DF11_E_INVALID_ARG),
    (dict(width=0), hdb.DF11_E_INVALID_ARG), (dict(ts=3), hdb.DF11_E_INVALID_ARG), (dict(width=1 << 28, ts=1 << 28), hdb.DF11_E_INVALID_ARG),
    (dict(batch=1 << 25), hdb.DF11_E_INVALID_ARG), (dict(width=4096, ts=4096), hdb.DF11_E_BUFFER_TOO_SMALL),
    (dict(width=4096, ts=4096, ws=P + 4, size=1 << 40), hdb.DF11_E_INVALID_ARG),
    (dict(width=4096, ts=4096, ws=None, size=1 << 40), hdb.DF11_E_INVALID_ARG),
])
def test_attention_refusals(change, status):
    a = dict(q=P, batch=2, heads=32, table=P, ts=4, width=4, lens=P, starts=None, out=P, lse=None, ws=None, size=0)
    a.update(change)
    c = cache()
    got = hdb.lib().df11_paged_attention(ctypes.byref(c), a["q"], a["batch"], a["heads"], 4096, 128, a["table"], a["ts"],
                                         a["width"], a["lens"], a["starts"], 1.0, a["out"], a["lse"], a["ws"], a["size"],
                                         None)
    assert got == status


def test_workspace_sizes():
    assert hdb.df11_mx4_matmul_workspace_bytes(1, 4096, 4096) == 0
    assert hdb.df11_mx4_matmul_workspace_bytes(3, 40, 63, False) == 0
    assert hdb.df11_mx4_matmul_workspace_bytes(4096, 4096, 64) == 0
    assert hdb.df11_mx4_matmul_workspace_bytes(4096, 4096, 63) >= 4096 * 64 * 2
    assert hdb.df11_mx4_matmul_workspace_bytes(4096, 4096, 64, False) >= 4096 * 64 * 2
    assert hdb.df11_paged_attention_workspace_bytes(1, 32, 8, 128, 16, 4) == 0
    assert hdb.df11_paged_attention_workspace_bytes(1, 32, 8, 128, 16, 4096) >= 32 * 130 * 4
    # calls that the operators refuse need none
    assert hdb.df11_paged_attention_workspace_bytes(1, 33, 8, 128, 16, 4096) == 0
    assert hdb.df11_paged_attention_workspace_bytes(1, 32, 8, 128, 17, 4096) == 0


class Streams:
    """torch as far as a call's place goes: GPU 0 with a current stream, and ExternalStream, which takes a handle of 0 for
    none and gives another stream."""

    def __init__(self, current):
        class Stream:
            def __init__(self, handle, device):
                self.cuda_stream, self.device_index = handle, device

        class ExternalStream(Stream):
            def __init__(self, handle, device=None):
                super().__init__(handle or 0xABC0, device)

        class cuda:
            pass

        cuda.Stream, cuda.ExternalStream = Stream, ExternalStream
        cuda.default_stream = staticmethod(lambda dev: Stream(0, dev))
        cuda.stream = staticmethod(lambda s: ("on", s.cuda_stream))
        cuda.device = staticmethod(lambda d: ("device", d))

        class _C:
            _cuda_getDevice = staticmethod(lambda: 0)
            _cuda_getCurrentRawStream = staticmethod(lambda dev: current)

        self.cuda, self._C = cuda, _C


@pytest.mark.parametrize("current", [0, 0x40])
@pytest.mark.parametrize("given", [None, 0, 0x40, 0x80])
@pytest.mark.parametrize("gpu", [0, 1])
def test_place_of_a_raw_handle(monkeypatch, current, given, gpu):
    """A call runs on the handle that it is given, the null stream's among them, and allocates there."""
    monkeypatch.setattr(hdb.step, "_torch", Streams(current))
    handle, ctx = hdb.step._place(gpu, given)
    want = current if given is None else given
    assert handle == want
    if given is None:
        assert ctx == (None if gpu == 0 else ("device", gpu))
    else:
        assert ctx == (None if gpu == 0 and given == current else ("on", want))


def test_a_derivative_is_refused():
    """What asks for a gradient or carries a tangent is told apart from what does not, on the CPU's tensors."""
    import torch
    from torch.autograd import forward_ad

    step = hdb.step
    step._torch or step._load()
    leaf, plain = torch.zeros(2, requires_grad=True), torch.zeros(2)
    for t in (leaf, leaf * 2):
        with pytest.raises(ValueError, match="an_entry has no backward"):
            step._no_gradient("an_entry", None, plain, t)
        step._no_gradient("an_entry", plain, t.detach())
        with torch.no_grad():
            step._no_gradient("an_entry", plain, t)
    with torch.inference_mode():
        step._no_gradient("an_entry", leaf)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(plain, torch.ones(2))
        step._no_gradient("an_entry", plain, None)
        for grad in (True, False):
            with torch.set_grad_enabled(grad), pytest.raises(ValueError, match="an_entry has no derivative"):
                step._no_gradient("an_entry", None, dual)


@pytest.mark.parametrize("change", [
    # more rows of w than a launch has work items for, with 1, 4, 5 and 32 rows of x, and more tiles than that
    dict(m=1, n=1 << 27), dict(m=4, n=(1 << 27) - 15), dict(m=1, n=(1 << 31) - 1), dict(m=5, n=1 << 29), dict(m=32, n=1 << 30),
    dict(m=1 << 19, n=1 << 20), dict(m=1 << 31 - 1, n=1 << 31 - 1),
    # rows of x or y past 2^48 values
    dict(m=1 << 20, xs=1 << 32), dict(m=1 << 20, n=64, ys=1 << 32),
])
def test_products_past_a_launch_or_the_addresses(change):
    a = dict(x=P, m=3, k=64, xs=64, codes=P, scales=P, n=40, y=P, ws=P, size=1 << 62)
    a.update(change)
    ys = a.get("ys", a["n"])
    L = hdb.lib()
    assert L.df11_mx4_matmul(a["x"], a["m"], a["k"], a["xs"], a["codes"], a["scales"], a["n"], a["y"], ys, a["ws"], a["size"],
                             None) == hdb.DF11_E_INVALID_ARG
    if "xs" not in change and "ys" not in change:
        assert hdb.df11_mx4_matmul_workspace_bytes(a["m"], a["n"], 63, False) == 0


@pytest.mark.parametrize("change", [
    dict(n_pages=1 << 30, k_page_stride=1 << 18), dict(n_pages=(1 << 31) - 1, v_page_stride=1 << 40),
    dict(kv_heads=1 << 16, k_head_stride=1 << 32), dict(page_size=1024, v_row_stride=1 << 38),
    dict(n_pages=1 << 29, k_page_stride=1 << 18, kv_heads=1 << 15, k_head_stride=1 << 32),  # half of it each
])
def test_caches_past_the_addresses(change):
    L = hdb.lib()
    c = cache(**change)
    heads = c.kv_heads
    assert L.df11_paged_append(ctypes.byref(c), P, 1024, 128, P, 1024, 128, P, 1, None) == hdb.DF11_E_INVALID_ARG
    assert L.df11_paged_attention(ctypes.byref(c), P, 1, heads, 1024, 128, P, 4, 4, P, None, 1.0, P, P, P, 1 << 62, None) == \
        hdb.DF11_E_INVALID_ARG


@pytest.mark.parametrize("change", [dict(tokens=1 << 30, ks=1 << 18), dict(tokens=1 << 30, vs=1 << 40), dict(kh=1 << 40, kv_heads=256),
                                    dict(vh=1 << 40, kv_heads=256)])
def test_appends_past_the_addresses(change):
    a = dict(tokens=1, ks=1024, kh=128, vs=1024, vh=128, kv_heads=8)
    a.update(change)
    c = cache(kv_heads=a["kv_heads"])
    assert hdb.lib().df11_paged_append(ctypes.byref(c), P, a["ks"], a["kh"], P, a["vs"], a["vh"], P, a["tokens"], None) == \
        hdb.DF11_E_INVALID_ARG


@pytest.mark.parametrize("change", [
    # workgroups: a cache head of a sequence each, cut into chunks, and rows of the join
    dict(batch=1 << 21), dict(batch=1 << 24), dict(batch=1 << 17, heads=128, kv_heads=128), dict(batch=1 << 20, width=512),
    dict(batch=1 << 19, heads=32, kv_heads=2, width=512),
    # addresses
    dict(batch=1 << 15, qb=1 << 33), dict(heads=1 << 20, qh=1 << 40), dict(batch=1 << 15, ts=1 << 33),
])
def test_attention_past_a_launch_or_the_addresses(change):
    a = dict(batch=2, heads=8, kv_heads=8, qb=4096, qh=128, width=4)
    a.update(change)
    c = cache(kv_heads=a["kv_heads"])
    got = hdb.lib().df11_paged_attention(ctypes.byref(c), P, a["batch"], a["heads"], a["qb"], a["qh"], P, a.get("ts", a["width"]),
                                         a["width"], P, None, 1.0, P, None, P, 1 << 62, None)
    assert got == hdb.DF11_E_INVALID_ARG
    if not {"qb", "qh", "ts"} & set(change):
        assert hdb.df11_paged_attention_workspace_bytes(a["batch"], a["heads"], a["kv_heads"], 128, 16, a["width"]) == 0


def test_a_stream_of_another_gpu_is_refused(monkeypatch):
    fake = Streams(0x40)
    monkeypatch.setattr(hdb.step, "_torch", fake)
    assert hdb.step._place(1, fake.cuda.Stream(0x80, 1)) == (0x80, ("on", 0x80))
    with pytest.raises(ValueError, match="GPU 0, the tensors to 1"):
        hdb.step._place(1, fake.cuda.Stream(0x80, 0))
