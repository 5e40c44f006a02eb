"""Host-only checks of the large products' entry points: invalid arguments return their status before any CUDA call
(fake, never-dereferenced data pointers), plans report the same, and the Python calls refuse what they cannot take."""
import ctypes

import pytest
import torch

import segmented_gather_gemm_expand_b200 as sg
from segmented_gather_gemm_expand_b200 import _abi

FAKE = 0x10000
T, K, N, R, A, B = 20, 64, 96, 16, 3, 4


def mk(shape, dt=_abi.BF16, data=FAKE, strides=None):
    if strides is None:
        strides, s = [], 1
        for n in reversed(shape):
            strides.insert(0, s)
            s *= max(n, 1)
    return _abi.make_tensor(data, dt, shape, strides)


def meta():
    return dict(s=mk((B,), _abi.I64), l=mk((B,), _abi.I32), i=mk((B,), _abi.I32), batches=B, longest=7)


def lora(**over):
    a = dict(x=mk((T, K)), w=mk((N, K)), bias=None, a=mk((A, R, K)), b=mk((A, N, R)), out=mk((T, N)), ws=FAKE, wsb=1 << 20, **meta())
    a.update(over)
    return a


def ref(t):
    return None if t is None else ctypes.byref(t)


def call_lora(a):
    return _abi.load().sgmv_lora_linear(*[ref(a[k]) for k in ("x", "w", "bias", "a", "b", "out", "s", "l", "i")], a["batches"], a["longest"],
                                        a["ws"], a["wsb"], None)


def plan_lora(a):
    v, n, p = ctypes.c_int(-1), ctypes.c_size_t(9), ctypes.c_size_t(9)
    rc = _abi.load().sgmv_lora_linear_plan(*[ref(a[k]) for k in ("x", "w", "bias", "a", "b", "out", "s", "l", "i")], a["batches"], a["longest"],
                                           ctypes.byref(v), ctypes.byref(n), ctypes.byref(p))
    return rc, v.value, n.value, p.value


META_BAD = {
    "meta_dtype": (dict(s=mk((B,), _abi.F16)), "SGMV_ERR_DTYPE"),
    "meta_2d": (dict(l=mk((B, 1), _abi.I32)), "SGMV_ERR_NDIM"),
    "meta_short": (dict(batches=B + 1), "SGMV_ERR_BATCHES"),
    "meta_null": (dict(i=mk((B,), _abi.I32, 0)), "SGMV_ERR_NULL_ARG"),
    "negative_batches": (dict(batches=-1), "SGMV_ERR_BATCHES"),
    "negative_longest": (dict(longest=-1), "SGMV_ERR_SHAPE"),
}
LORA_BAD = {
    "x_dtype": (dict(x=mk((T, K), _abi.I32)), "SGMV_ERR_DTYPE"),
    "w_dtype_f32": (dict(w=mk((N, K), _abi.F32)), "SGMV_ERR_DTYPE"),
    "a_dtype_differs": (dict(a=mk((A, R, K), _abi.F16)), "SGMV_ERR_DTYPE"),
    "b_dtype_differs": (dict(b=mk((A, N, R), _abi.F16)), "SGMV_ERR_DTYPE"),
    "bias_dtype_differs": (dict(bias=mk((N,), _abi.F32)), "SGMV_ERR_DTYPE"),
    "out_dtype": (dict(out=mk((T, N), _abi.I64)), "SGMV_ERR_DTYPE"),
    "w_3d": (dict(w=mk((1, N, K))), "SGMV_ERR_NDIM"),
    "a_2d": (dict(a=mk((R, K))), "SGMV_ERR_NDIM"),
    "bias_2d": (dict(bias=mk((1, N))), "SGMV_ERR_NDIM"),
    "w_k": (dict(w=mk((N, K + 8))), "SGMV_ERR_RANK_MISMATCH"),
    "a_k": (dict(a=mk((A, R, K + 8))), "SGMV_ERR_RANK_MISMATCH"),
    "b_rank": (dict(b=mk((A, N, R + 8))), "SGMV_ERR_RANK_MISMATCH"),
    "b_n": (dict(b=mk((A, N + 8, R))), "SGMV_ERR_SLICE_SIZE"),
    "adapter_counts": (dict(b=mk((A + 1, N, R))), "SGMV_ERR_SHAPE"),
    "bias_length": (dict(bias=mk((N + 1,))), "SGMV_ERR_SHAPE"),
    "out_width": (dict(out=mk((T, N + 8))), "SGMV_ERR_OUT_WIDTH"),
    "a_4d": (dict(a=mk((A, 2, R, K))), "SGMV_ERR_LAYOUT_4D"),
    "b_4d": (dict(b=mk((A, 2, N, R))), "SGMV_ERR_LAYOUT_4D"),
    "out_turned": (dict(out=mk((T, N), strides=(1, T))), "SGMV_ERR_OUT_NOT_CONTIGUOUS"),
    "out_rows_overlap": (dict(out=mk((T, N), strides=(N - 1, 1))), "SGMV_ERR_OUT_NOT_CONTIGUOUS"),
    "null_x": (dict(x=mk((T, K), data=0)), "SGMV_ERR_NULL_ARG"),
    "negative_stride": (dict(w=mk((N, K), strides=(-K, 1))), "SGMV_ERR_STRIDE"),
    "huge_rank": (dict(a=mk((A, 1 << 21, K)), b=mk((A, N, 1 << 21))), "SGMV_ERR_TOO_LARGE"),
    **META_BAD,
}


@pytest.mark.parametrize("case", sorted(LORA_BAD))
def test_lora_linear_refuses(case):
    over, code = LORA_BAD[case]
    a = lora(**over)
    assert call_lora(a) == _abi.STATUS[code]
    assert plan_lora(a) == (_abi.STATUS[code], 0, 0, 0)


@pytest.mark.parametrize("over", [dict(ws=None), dict(ws=FAKE + 8), dict(wsb=100)])
def test_lora_linear_refuses_workspaces(over):
    assert call_lora(lora(**over)) == _abi.STATUS["SGMV_ERR_WORKSPACE"]


@pytest.mark.parametrize("over", [dict(x=mk((0, K), data=0)), dict(w=mk((0, K), data=0), b=mk((A, 0, R), data=0), out=mk((T, 0), data=0))])
def test_lora_linear_empty(over):
    assert call_lora(lora(**over)) == 0


def grouped(name, **over):
    if name == "sgmv_grouped_gemm":
        a = dict(a=mk((T, K)), b=mk((A, N, K)), c=mk((T, N)), **meta())
    else:
        a = dict(a=mk((T, N)), b=mk((T, K)), c=mk((A, N, K)), **meta())
    a.update(over)
    return a


def call_grouped(name, a, add=0):
    return getattr(_abi.load(), name)(*[ref(a[k]) for k in ("a", "b", "c", "s", "l", "i")], a["batches"], a["longest"], add, None)


GROUPED_BAD = {
    ("sgmv_grouped_gemm", "x_dtype"): (dict(a=mk((T, K), _abi.I32)), "SGMV_ERR_DTYPE"),
    ("sgmv_grouped_gemm", "w_f32"): (dict(b=mk((A, N, K), _abi.F32)), "SGMV_ERR_DTYPE"),
    ("sgmv_grouped_gemm", "w_2d"): (dict(b=mk((N, K))), "SGMV_ERR_NDIM"),
    ("sgmv_grouped_gemm", "w_4d"): (dict(b=mk((A, 2, N, K))), "SGMV_ERR_LAYOUT_4D"),
    ("sgmv_grouped_gemm", "k"): (dict(b=mk((A, N, K + 8))), "SGMV_ERR_RANK_MISMATCH"),
    ("sgmv_grouped_gemm", "out_width"): (dict(c=mk((T, N + 8))), "SGMV_ERR_OUT_WIDTH"),
    ("sgmv_grouped_gemm", "out_turned"): (dict(c=mk((T, N), strides=(1, T))), "SGMV_ERR_OUT_NOT_CONTIGUOUS"),
    ("sgmv_grouped_gemm", "null_w"): (dict(b=mk((A, N, K), data=0)), "SGMV_ERR_NULL_ARG"),
    ("sgmv_grouped_wgrad", "dy_dtype"): (dict(a=mk((T, N), _abi.I32)), "SGMV_ERR_DTYPE"),
    ("sgmv_grouped_wgrad", "dw_2d"): (dict(c=mk((N, K))), "SGMV_ERR_NDIM"),
    ("sgmv_grouped_wgrad", "dw_4d"): (dict(c=mk((A, 2, N, K))), "SGMV_ERR_LAYOUT_4D"),
    ("sgmv_grouped_wgrad", "k"): (dict(b=mk((T, K + 8))), "SGMV_ERR_RANK_MISMATCH"),
    ("sgmv_grouped_wgrad", "n"): (dict(a=mk((T, N + 8))), "SGMV_ERR_SLICE_SIZE"),
    ("sgmv_grouped_wgrad", "dw_turned"): (dict(c=mk((A, N, K), strides=(N * K, 1, N))), "SGMV_ERR_OUT_NOT_CONTIGUOUS"),
    ("sgmv_grouped_wgrad", "dw_overlaps"): (dict(c=mk((A, N, K), strides=(K, K, 1))), "SGMV_ERR_OUT_NOT_CONTIGUOUS"),
    ("sgmv_grouped_wgrad", "null_dy"): (dict(a=mk((T, N), data=0)), "SGMV_ERR_NULL_ARG"),
    **{(n, k): v for k, v in META_BAD.items() for n in ("sgmv_grouped_gemm", "sgmv_grouped_wgrad")},
}


@pytest.mark.parametrize("case", sorted(GROUPED_BAD))
def test_grouped_refuses(case):
    over, code = GROUPED_BAD[case]
    a = grouped(case[0], **over)
    assert call_grouped(case[0], a) == _abi.STATUS[code]
    v = ctypes.c_int(-1)
    rc = getattr(_abi.load(), case[0] + "_plan")(*[ref(a[k]) for k in ("a", "b", "c", "s", "l", "i")], a["batches"], a["longest"], 0,
                                                 ctypes.byref(v))
    assert (rc, v.value) == (_abi.STATUS[code], 0)


def test_grouped_empty():
    assert call_grouped("sgmv_grouped_gemm", grouped("sgmv_grouped_gemm", batches=0)) == 0
    assert call_grouped("sgmv_grouped_gemm", grouped("sgmv_grouped_gemm", a=mk((0, K), data=0))) == 0
    assert call_grouped("sgmv_grouped_wgrad", grouped("sgmv_grouped_wgrad", batches=0), add=1) == 0
    assert call_grouped("sgmv_grouped_wgrad", grouped("sgmv_grouped_wgrad", c=mk((0, N, K), data=0))) == 0


def test_null_descriptors():
    lib = _abi.load()
    a = grouped("sgmv_grouped_gemm")
    assert lib.sgmv_grouped_gemm(None, ref(a["b"]), ref(a["c"]), ref(a["s"]), ref(a["l"]), ref(a["i"]), B, 7, 0, None) == -1
    assert lib.sgmv_grouped_gemm_plan(*[ref(a[k]) for k in ("a", "b", "c", "s", "l", "i")], B, 7, 0, None) == -1
    assert call_lora(lora(a=None)) == -1


def test_python_calls_refuse_host_tensors_and_wrong_types():
    x, w, out, m = torch.zeros(4, 8), torch.zeros(2, 6, 8), torch.zeros(4, 6), [torch.zeros(2, dtype=torch.int32)] * 3
    with pytest.raises(ValueError):
        sg.sgmv_grouped_gemm(x, w, out, *m, 2, 2)
    with pytest.raises(ValueError):
        sg.sgmv_grouped_wgrad(out, x, w, *m, 2, 2)
    with pytest.raises(ValueError):
        sg.sgmv_lora_linear(x, w[0], w, w, out, *m, 2, 2)
    with pytest.raises(ValueError):
        sg.lora_linear_plan(x, w[0], w, w, out, *m, 2, 2)
    with pytest.raises(TypeError):
        sg.sgmv_grouped_gemm(x, w, None, *m, 2, 2)
