"""Host-side checks of the operators' entry points beyond their arguments' ranges (no GPU needed)."""
import ctypes as C

from mixed_precision_quantized_fp32_b200 import _lib
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
