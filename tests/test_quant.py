"""Refusals of the 4-bit product's entry points (include/moe_quant.h) and its
word format, on the CPU."""
import ctypes as C

import numpy as np
import pytest

from compressed_expert_ffn_amd import _lib as L


def create(n_in=64, n_out=48, group=32, x_dtype="f16", **w):
    cfg = L.moe_quant_config(n_in, n_out, group, L.DTYPE[x_dtype])
    ws = L.moe_quant_weights()
    for key, v in w.items():
        setattr(ws, key, v)
    h = C.c_void_p(1234)
    rc = L.lib.moe_quant_create(C.byref(cfg), C.byref(ws), None, C.byref(h))
    assert not h.value  # nothing is handed out on an error
    return rc, L.lib.moe_last_error().decode()


Q = np.zeros((64, 48), dtype=np.int8)
S = np.ones((2, 48), dtype=np.float16)
GIVEN = dict(q=Q.ctypes.data, scale=S.ctypes.data)

BAD = [
    (dict(n_in=0), L.MOE_ERR_INVALID_ARG, "positive"),
    (dict(n_out=-3), L.MOE_ERR_INVALID_ARG, "positive"),
    (dict(group=16), L.MOE_ERR_UNSUPPORTED, "group"),
    (dict(group=0), L.MOE_ERR_UNSUPPORTED, "group"),
    (dict(x_dtype="f32"), L.MOE_ERR_UNSUPPORTED, "F16 or BF16"),
    (dict(n_in=1 << 25), L.MOE_ERR_UNSUPPORTED, "2^24"),
    (dict(n_in=1 << 20, n_out=1 << 12), L.MOE_ERR_UNSUPPORTED, "2^31"),
    (dict(q=None), L.MOE_ERR_INVALID_ARG, "either"),
    (dict(values=Q.ctypes.data), L.MOE_ERR_INVALID_ARG, "either"),
    (dict(scale=None), L.MOE_ERR_INVALID_ARG, "scale"),
    (dict(q=None, values=Q.ctypes.data, values_dtype=7), L.MOE_ERR_INVALID_ARG, "values_dtype"),
]


@pytest.mark.parametrize("change,code,msg", BAD)
def test_create_refuses(change, code, msg):
    rc, text = create(**{**GIVEN, **change})
    assert rc == code and msg in text


def test_unknown_dtype_and_null_arguments():
    cfg = L.moe_quant_config(64, 48, 32, 9)
    ws, h = L.moe_quant_weights(), C.c_void_p()
    assert L.lib.moe_quant_create(C.byref(cfg), C.byref(ws), None, C.byref(h)) == L.MOE_ERR_INVALID_ARG
    cfg = L.moe_quant_config(64, 48, 32, 1)
    assert L.lib.moe_quant_create(None, C.byref(ws), None, C.byref(h)) == L.MOE_ERR_INVALID_ARG
    assert L.lib.moe_quant_create(C.byref(cfg), None, None, C.byref(h)) == L.MOE_ERR_INVALID_ARG
    assert L.lib.moe_quant_create(C.byref(cfg), C.byref(ws), None, None) == L.MOE_ERR_INVALID_ARG
    assert L.lib.moe_quant_matvec(None, None, 64, 1, None, 48, None) == L.MOE_ERR_INVALID_ARG
    assert L.lib.moe_quant_read(None, None, None) == L.MOE_ERR_INVALID_ARG
    assert L.lib.moe_quant_bytes(None) == 0
    assert L.lib.moe_quant_destroy(None) == L.MOE_OK


@pytest.mark.parametrize("kw,msg", [
    (dict(q=Q[:32], scale=S), "shape"),
    (dict(q=Q, scale=S[:1]), "shape"),
    (dict(q=Q.astype(np.int32), scale=S), "dtype"),
    (dict(q=Q, scale=S.astype(np.float32)), "dtype"),
    (dict(values=Q), "dtype"),
])
def test_binding_refuses_wrong_arrays(kw, msg):
    with pytest.raises(ValueError, match=msg):
        L.QuantLinear(64, 48, 32, "f16", **kw)


def test_binding_refuses_a_host_tensor_as_rows():
    import torch
    lin = L.QuantLinear.__new__(L.QuantLinear)
    lin.h, lin.n_in, lin.n_out, lin.group, lin.dtype, lin.device = None, 64, 48, 32, torch.float16, 0
    with pytest.raises(ValueError, match="device"):
        lin.matvec(torch.zeros((1, 64), dtype=torch.float16))
    with pytest.raises(ValueError, match=r"\[T, 64\]"):
        lin.matvec(torch.zeros((1, 63), dtype=torch.float16))
    with pytest.raises(ValueError, match="torch.float16"):
        lin.matvec(torch.zeros((1, 64)))
