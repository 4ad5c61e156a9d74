"""Host-side checks of the operators' entry points beyond their arguments' ranges (no GPU needed)."""
import ctypes as C
import importlib.metadata
import os

import pytest
import torch

import mixed_precision_quantized_fp32_b200 as moe
from mixed_precision_quantized_fp32_b200 import _lib
from mixed_precision_quantized_fp32_b200 import build as bld
from tests.test_ops_host import ARGS, FAKE, OK, no_gpu


# ------------------------------------------------------------------ the entry with test hooks
def debug_call(dbg=None, **change):
    a = dict(ARGS["moe_adapters"], **change)
    a.pop("status")
    return _lib.STATUS[_lib.load().moe_adapters_debug(*a.values(), dbg, None)]


def test_adapters_debug_refuses_what_adapters_refuses():
    assert debug_call(x=None) == "MOE_ERR_ARG" and debug_call(r=12) == "MOE_ERR_SHAPE"
    assert debug_call(dtype=2) == "MOE_ERR_FORMAT" and debug_call(B=FAKE + 8) == "MOE_ERR_ALIGN"
    assert debug_call(C.byref(_lib.MoeDebug(status=FAKE + 2))) == "MOE_ERR_ALIGN"


@no_gpu
def test_adapters_debug_without_hooks_reaches_the_device_check():
    assert debug_call() in OK and debug_call(C.byref(_lib.MoeDebug(status=FAKE))) in OK


# ------------------------------------------------------------------ what the binding's object is built of
def test_binding_is_rebuilt_when_torch_python_or_the_command_change(tmp_path, monkeypatch):
    # it is compiled against internal headers of torch and Python: an object of other versions may not load
    lib = str(tmp_path / "bind.so")
    ran = []

    def compile_(cmd, check):
        ran.append(cmd)
        open(lib + ".tmp", "w").close()

    monkeypatch.setattr(bld, "BIND_LIB", lib)
    monkeypatch.setattr(bld, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(bld.subprocess, "run", compile_)

    def runs():
        ran.clear()
        assert bld.build_bind() == lib and os.path.exists(lib)
        return len(ran)

    assert runs() == 1 and runs() == 0
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0" if name == "torch" else version(name))
    assert runs() == 1 and runs() == 0
    monkeypatch.setattr(bld.sys, "version", "another Python")
    assert runs() == 1 and runs() == 0
    monkeypatch.setattr(bld, "NVCC", "/elsewhere/bin/nvcc")        # other headers
    assert runs() == 1 and runs() == 0
    os.utime(lib, (1, 1))                                          # older than its source
    assert runs() == 1


# ------------------------------------------------------------------ tensors that are more than their memory
T, K2, E, H = 4, 2, 3, 8


def calls():
    """Every call with its arguments by name, all tensors on the CPU (which each call refuses by itself)."""
    x, i, w = torch.zeros(T, H), torch.zeros(T, K2, dtype=torch.int32), torch.zeros(T, K2)
    r = moe.Routes(T, K2, E, i[:, 0], i[:, 0], i[:, 0])
    c = moe.ActCkpt(torch.zeros(T, H, dtype=torch.int8), torch.zeros(T, 1, dtype=torch.uint8), torch.float32)
    return {
        "dispatch": (lambda x: moe.moe_dispatch(x, i, E), dict(x=x)),
        "dispatch_backward": (lambda dxs: moe.moe_dispatch_backward(dxs, r), dict(dxs=x)),
        "collect": (lambda o: moe.moe_collect(o, w, r), dict(o=x)),
        "collect_backward": (lambda dy, o: moe.moe_collect_backward(dy, o, w, r), dict(dy=x, o=x)),
        "act_save": (lambda x: moe.moe_act_save(x), dict(x=x)),
        "swiglu_save": (lambda g, u: moe.moe_swiglu_save(g, u), dict(g=x, u=x)),
        "swiglu_backward": (lambda dh: moe.moe_swiglu_backward(dh, moe.SwigluCkpt(c, c)), dict(dh=x)),
        "adapters": (lambda x, y, A, B: moe.moe_adapters(x, y, A, B, w[:, 0], r), dict(x=x, y=x, A=x, B=x)),
    }


@pytest.mark.parametrize("name", calls())
def test_lazily_negated_views_are_refused(name):
    call, args = calls()[name]
    with pytest.raises(ValueError, match="cuda"):
        call(**args)
    for key in args:
        with pytest.raises(ValueError, match=f"{key} is negated"):
            call(**dict(args, **{key: torch._neg_view(args[key])}))


@pytest.mark.parametrize("name", calls())
def test_tensors_that_take_part_in_a_gradient_are_refused_where_it_would_be_lost(name):
    import torch.autograd.forward_ad as fwd
    call, args = calls()[name]
    for key in args:
        leaf = dict(args, **{key: args[key].clone().requires_grad_()})
        inner = dict(args, **{key: leaf[key] * 2})
        for a in (leaf, inner):
            with pytest.raises(ValueError, match=f"{key} takes part in a gradient"):
                call(**a)
            for quiet in (torch.no_grad, torch.inference_mode):
                with quiet(), pytest.raises(ValueError, match="cuda"):     # as without one
                    call(**a)
        with fwd.dual_level():
            dual = fwd.make_dual(args[key], torch.ones_like(args[key]))
            with pytest.raises(ValueError, match=f"{key} takes part in a gradient"):
                call(**dict(args, **{key: dual}))
        with pytest.raises(ValueError, match="cuda"):
            call(**dict(args, **{key: leaf[key].detach()}))


def test_the_body_of_an_autograd_function_is_not_refused():
    call, args = calls()["collect"]

    class Collect(torch.autograd.Function):
        @staticmethod
        def forward(ctx, o):
            with pytest.raises(ValueError, match="cuda"):
                call(o=o)
            return o.clone()

        @staticmethod
        def backward(ctx, g):
            with pytest.raises(ValueError, match="cuda"):
                call(o=g)
            return g

    o = args["o"].clone().requires_grad_()
    Collect.apply(o).sum().backward()
    assert torch.equal(o.grad, torch.ones_like(o))
