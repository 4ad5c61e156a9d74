"""Host-side checks of the operators around the expert products (no GPU needed): sizes,
and refusals before anything is launched.  Pointers are fake device addresses."""
import ctypes as C

import pytest
import torch

import mixed_precision_quantized_fp32_b200 as moe
from mixed_precision_quantized_fp32_b200 import _lib

FAKE = 0x7F0000000000  # 256-byte aligned, never dereferenced
NAMES = ("moe_sort", "moe_dispatch", "moe_dispatch_backward", "moe_collect", "moe_collect_backward", "moe_act_save",
         "moe_act_load", "moe_swiglu_save", "moe_swiglu_backward", "moe_adapters")
OK = ("MOE_ERR_CUDA", "MOE_ERR_UNSUPPORTED_DEVICE")  # a valid call where there is no device
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the fake pointers would be launched on")

# arguments by name, in the order of the declarations, with values that are accepted
ARGS = {
    "moe_sort": dict(idx=FAKE, T=16, k=2, E=8, perm=FAKE, inv=FAKE, offsets=FAKE, ws=FAKE, ws_bytes=1 << 20, need=None),
    "moe_dispatch": dict(x=FAKE, ldx=64, dtype=0, idx=FAKE, T=16, k=2, E=8, H=64, xs=FAKE, ldxs=64, perm=FAKE, inv=FAKE,
                         offsets=FAKE, ws=FAKE, ws_bytes=1 << 20, need=None),
    "moe_dispatch_backward": dict(dxs=FAKE, lddxs=64, dtype=0, inv=FAKE, T=16, k=2, H=64, dx=FAKE, lddx=64),
    "moe_collect": dict(o=FAKE, ldo=64, dtype=0, w=FAKE, inv=FAKE, T=16, k=2, H=64, y=FAKE, ldy=64),
    "moe_collect_backward": dict(dy=FAKE, lddy=64, o=FAKE, ldo=64, dtype=0, w=FAKE, inv=FAKE, T=16, k=2, H=64, d_o=FAKE,
                                 lddo=64, dw=FAKE),
    "moe_act_save": dict(x=FAKE, ldx=64, dtype=0, R=16, F=64, codes=FAKE, exps=FAKE, n_rows=None),
    "moe_act_load": dict(codes=FAKE, exps=FAKE, R=16, F=64, dtype=0, x=FAKE, ldx=64, n_rows=None),
    "moe_swiglu_save": dict(g=FAKE, ldg=64, u=FAKE, ldu=64, dtype=0, R=16, F=64, h=FAKE, ldh=64, gq=FAKE, ge=FAKE,
                            uq=FAKE, ue=FAKE, n_rows=None),
    "moe_swiglu_backward": dict(dh=FAKE, lddh=64, dtype=0, gq=FAKE, ge=FAKE, uq=FAKE, ue=FAKE, R=16, F=64, dg=FAKE,
                                lddg=64, du=FAKE, lddu=64, h=FAKE, ldh=64, n_rows=None),
    "moe_adapters": dict(x=FAKE, ldx=64, y=FAKE, ldy=64, dtype=0, T=16, K=64, N=64, r=16, n=4, A=FAKE, B=FAKE, scale=FAKE,
                         perm=FAKE, offsets=FAKE, out=FAKE + 65536, ldo=64, status=None),
}


def call(name, **change):
    a = dict(ARGS[name], **change)
    assert set(change) <= set(ARGS[name])
    return _lib.STATUS[getattr(_lib.load(), name)(*a.values(), None)]


def need(name, **change):
    n = C.c_uint64(0)
    assert call(name, ws=None, ws_bytes=0, need=C.byref(n), **change) == "MOE_OK"
    return n.value


@no_gpu
@pytest.mark.parametrize("name", NAMES)
def test_accepted_arguments_reach_the_device_check(name):
    assert call(name) in OK
    for dtype in (1, 2):
        if "dtype" in ARGS[name] and not (name == "moe_adapters" and dtype == 2):
            assert call(name, dtype=dtype) in OK


@pytest.mark.parametrize("name", NAMES)
def test_null_pointers_and_types(name):
    for key, v in ARGS[name].items():
        if v is not None and v in (FAKE, FAKE + 65536):
            if (name, key) in (("moe_swiglu_backward", "h"), ("moe_sort", "ws"), ("moe_dispatch", "ws")):
                continue                          # nullable (ws: a sort of few entries needs none)
            assert call(name, **{key: None}) == "MOE_ERR_ARG", key
    if "dtype" in ARGS[name]:
        for bad in (-1, 3, 16):
            assert call(name, dtype=bad) == "MOE_ERR_FORMAT"


@pytest.mark.parametrize("name", NAMES)
def test_shapes(name):
    a = ARGS[name]
    bad = {"T": (-1, 1 << 21), "k": (0, 9, -2), "E": (0, 1025, -1), "H": (0, -5, (1 << 20) + 1), "R": (-1,),
           "F": (0, -1, (1 << 20) + 1), "K": (0, 12, -8), "N": (0, 4, 12, -8), "r": (0, 4, 12, 136, -8), "n": (0, 1025, -1)}
    for key, values in bad.items():
        for v in values if key in a else ():
            assert call(name, **{key: v}) == "MOE_ERR_SHAPE", (key, v)
    for key in a:
        if key.startswith("ld"):
            assert call(name, **{key: 63}) == "MOE_ERR_SHAPE", key
    if "R" in a:                                   # R * groups beyond 31 bits
        wide = {k: 1 << 20 for k in a if k.startswith("ld")}
        assert call(name, R=1 << 16, F=1 << 20, **wide) == "MOE_ERR_SHAPE"
    if "k" in a:
        assert call(name, T=(1 << 20) // 2 + 1) == "MOE_ERR_SHAPE"


@pytest.mark.parametrize("name", NAMES)
def test_alignment(name):
    a = ARGS[name]
    for key in ("idx", "perm", "inv", "offsets", "w", "dw", "scale"):
        if key in a:
            assert call(name, **{key: FAKE + 2}) == "MOE_ERR_ALIGN", key
    for key in ("x", "xs", "dxs", "dx", "o", "y", "dy", "d_o", "g", "u", "h", "dh", "dg", "du"):
        if key in a:
            assert call(name, **{key: FAKE + 1}) == "MOE_ERR_ALIGN", key
            if name != "moe_adapters":
                assert call(name, **{key: FAKE + 2, "dtype": 2}) == "MOE_ERR_ALIGN", key
    if "n_rows" in a:
        assert call(name, n_rows=FAKE + 2) == "MOE_ERR_ALIGN"
    if "ws" in a:
        assert call(name, ws=FAKE + 128) == "MOE_ERR_ALIGN"
    if name == "moe_adapters":
        assert call(name, status=FAKE + 2) == "MOE_ERR_ALIGN"
        for key in ("x", "y", "A", "B", "out"):
            assert call(name, **{key: FAKE + 8}) == "MOE_ERR_ALIGN", key
        for key in ("ldx", "ldy", "ldo"):
            assert call(name, **{key: 68}) == "MOE_ERR_ALIGN", key


@pytest.mark.parametrize("name,big", [("moe_sort", dict(T=40000)), ("moe_dispatch", dict(T=40000))])
def test_workspaces(name, big):
    n = need(name, **big)
    assert n >= 256 and n % 256 == 0
    assert call(name, ws_bytes=n - 1, **big) == "MOE_ERR_WORKSPACE"
    assert need(name) <= n
    assert need(name, T=8192) == 0 and need(name, T=8193) > 0   # few entries: no workspace
    assert torch.cuda.is_available() or call(name, T=8192, ws=None, ws_bytes=0) in OK
    assert call(name, ws=None, need=None, **big) == "MOE_ERR_ARG"


def test_workspace_bounds():
    # one histogram of E+1 counts per block of the sort, at most 128 blocks
    for T, k, E in ((1, 1, 1), (1024, 1, 1024), (513, 2, 256), (1 << 20, 1, 1024), (131072, 8, 256)):
        assert need("moe_sort", T=T, k=k, E=E) <= 128 * (E + 1) * 4 + 256


@no_gpu
def test_empty_batches():
    for name in ("moe_dispatch_backward", "moe_collect", "moe_collect_backward"):
        assert call(name, T=0) == "MOE_OK"
    for name in ("moe_act_save", "moe_act_load", "moe_swiglu_save", "moe_swiglu_backward"):
        assert call(name, R=0) == "MOE_OK"
    assert call("moe_adapters", T=0) == "MOE_OK"
    # a sort of nothing still writes its offsets
    assert call("moe_sort", T=0, idx=None, perm=None, inv=None) in OK


def test_adapters_in_place_needs_one_pitch():
    assert call("moe_adapters", out=FAKE, y=FAKE, ldy=72) == "MOE_ERR_ARG"


def test_binding_refuses_cpu_tensors():
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    c = moe.ActCkpt(torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4, 1, dtype=torch.uint8), torch.float32)
    for codes, exps in ((x, c.exps), (c.codes, c.codes), (c.codes, torch.zeros(4, 2, dtype=torch.uint8)), (c.codes.T, c.exps)):
        with pytest.raises(ValueError):
            moe.ActCkpt(codes, exps, torch.float32)
    r = moe.Routes(4, 2, 3, i[:, 0], i[:, 0], i[:, 0])
    for f in (lambda: moe.moe_sort(i, 3), lambda: moe.moe_dispatch(x, i, 3), lambda: moe.moe_dispatch_backward(x, r),
              lambda: moe.moe_collect(x, x, r), lambda: moe.moe_collect_backward(x, x, x, r), lambda: moe.moe_act_save(x),
              lambda: moe.moe_act_load(c), lambda: moe.moe_swiglu_save(x, x),
              lambda: moe.moe_swiglu_backward(x, moe.SwigluCkpt(c, c)), lambda: moe.moe_adapters(x, x, x, x, x, r)):
        with pytest.raises(ValueError, match="cuda"):
            f()


def test_exports_cover_the_operators():
    assert set(NAMES) <= set(_lib.EXPORTS) and all(hasattr(_lib.load(), n) for n in NAMES)
    assert set(NAMES) <= set(moe.__all__)
