"""The binding's argument checks where they meet what is absurd: sizes past 64
bits.  In C++ and in Python alike (no GPU needed)."""
import pytest
import torch

import combine_ep_get_dispatch_amd as M
from combine_ep_get_dispatch_amd import binding as B
from test_checks import BOTH, x


@pytest.mark.parametrize("cls", BOTH)
def test_sizes_past_64_bits(cls):
    A = cls("some_call")
    with pytest.raises(M.MoeDispError, match=f"needs {2 ** 63}"):
        A.arg("x", x, B._ROWS_BF16, 2 ** 63)
    with pytest.raises(M.MoeDispError, match="x is required"):
        A.arg("x", None, B._ROWS_BF16, 2 ** 80)
    assert A.arg("x", x, B._ROWS_BF16, -2 ** 80) == x.data_ptr()


def test_calls_of_absurd_shapes():
    rows = M.moedisp_rows.contiguous(2 ** 31 - 1, 4)
    bounds, ws = torch.zeros(5, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    w = torch.zeros(8, 8)
    rows_bf16 = torch.zeros(8, dtype=torch.bfloat16)
    huge = 2 ** 31 - 1
    router = M.moedisp_router.make(huge, huge, huge)
    for call in (lambda: M.ep_expert_wgrad_bf16(rows, huge, huge, rows_bf16, rows_bf16, bounds, w, M.FP32, False, ws),
                 lambda: M.ep_expert_gemm_bf16(rows, huge, huge, 0, rows_bf16, rows_bf16, bounds, w, M.FP32, ws),
                 lambda: M.ep_expert_gemm_w4(rows, huge, huge, 0, rows_bf16, ws, ws, bounds, w, M.FP32, ws),
                 lambda: M.ep_router_topk(router, w, None, None, bounds, w)):
        with pytest.raises(M.MoeDispError):
            call()


@pytest.mark.parametrize("cls", BOTH)
def test_size_of_a_weight_gradient(cls):
    """E * N * K * 4 with each at its type's largest is past 2^63."""
    A = cls("ep_expert_wgrad_bf16")
    with pytest.raises(M.MoeDispError, match="dw holds"):
        A.arg("dw", torch.zeros(8, 8), B._F32, (2 ** 31 - 1) ** 3 * 4, written=True)


def test_integers_past_32_bits():
    """ctypes would cut them off: FP32 + 2^32 would be checked as bf16 results
    and written as binary32, and 256 - 2^32 channels need no memory here."""
    past, cut = 2 ** 32, -2 ** 32
    r = M.moedisp_rows.contiguous(1, 4)
    t = torch.zeros(0)
    for call in (lambda v: M.ep_expert_gemm(r, 256, 256, 0, t, t, t, t, t, t, M.FP32 + v, t),
                 lambda v: M.ep_expert_gemm(r, 256, 256 + v, 0, t, t, t, t, t, t, M.FP32, t),
                 lambda v: M.ep_expert_wgrad(r, 256 + v, 256, 0, t, t, t, t, t, M.FP32, False, t),
                 lambda v: M.ep_swiglu_quant(r, 256 + v, 0, t, t, t, t, t),
                 lambda v: M.ep_swiglu_backward(r, 256, v, t, t, t, t, t, t, t),
                 lambda v: M.ep_swiglu(r, 256 + v, t, t, t, t),
                 lambda v: M.ep_expert_gemm_bf16(r, 256, 256, 1 + v, t, t, t, t, M.FP32, t),
                 lambda v: M.ep_expert_gemm_bf16(r, 256, 256, 1, t, t, t, t, M.FP32 + v, t),
                 lambda v: M.ep_expert_wgrad_bf16(r, 256, 256 + v, t, t, t, t, M.FP32, False, t),
                 lambda v: M.ep_expert_gemm_w4(r, 256, 256, M.W4_INT4 + v, t, t, t, t, t, M.FP32, t)):
        for v in (past, cut):
            with pytest.raises(M.MoeDispError, match="32 bits"):
                call(v)
    shape = M.moedisp_shape.make(4, 256, 4, 2, 2)
    for call in (lambda v: M.ep_combine(shape, t, t, t, t, t, M.FP32 + v, t),
                 lambda v: M.ep_combine_padded(shape, 4 + v, t, t, t, t, t, M.FP32, t),
                 lambda v: M.ep_combine_groups(shape, t, t, t, t, M.FP32 + v, t),
                 lambda v: M.ep_group_reduce(shape, t, t, t, t, t, t, M.FP32 + v, t),
                 lambda v: M.ep_dispatch_quant(shape, 128, 1 + v, *[t] * 11),
                 lambda v: M.ep_layout_dispatch_small_padded(shape, 4, 4 + v, 0, *[t] * 13)):
        for v in (past, cut):
            with pytest.raises(M.MoeDispError, match="32 bits"):
                call(v)


def test_probes_of_negative_sizes():
    t = torch.zeros(64)
    for call in (lambda: M.ep_probe_read(t, -16, t), lambda: M.ep_probe_copy(t, t, -16), lambda: M.ep_probe_fill(t, -4096)):
        with pytest.raises(M.MoeDispError, match="negative"):
            call()


@pytest.mark.parametrize("cls", BOTH)
def test_misuse_raises_alike(cls):
    """Calls that the binding itself never makes: TypeError in both forms, and
    no more tensors than a call has."""
    A = cls("c")
    for bad in (("x",), ("x", x, None, "many"), ("x", None, None, "many", True), ("x", x, None, 1.5),
                ("x", x, [torch.bfloat16], 1), ("x", x, torch.bfloat16, 1), ("x", x, None, 1, False, False, 1)):
        with pytest.raises(TypeError):
            A.arg(*bad)
    with pytest.raises(TypeError):
        A.arg("x", x, None, 1, wrong=True)
    for _ in range(24):
        A.arg("x", x, None, 1)
    A.arg("none", None, None, 1, True)
    with pytest.raises(TypeError):
        A.arg("x", x, None, 1)
