"""Argument checks of the bf16 and 4-bit products, the bf16 activation and the
router's choice (no GPU needed): every call below is rejected on the host, with
the documented code, before anything touches a device."""
import ctypes as C
import math
import os

import pytest
import torch

import combine_ep_get_dispatch_amd as M
from combine_ep_get_dispatch_amd import binding as B
from test_experts_abi import BAD_ROWS, NULL, p, rows


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from combine_ep_get_dispatch_amd import build
        build.build()
    return M.load()


def gemm(lib, r=None, n=256, k=256, lay=0, x=None, w=None, b=None, y=None, dt=M.BF16, ws=None, nws=256):
    return lib.ep_expert_gemm_bf16(C.byref(r or rows()), n, k, lay, x or p(), w or p(), b or p(), y or p(), dt,
                                   ws or p(), nws, None)


def wgrad(lib, r=None, n=256, k=256, x=None, dy=None, b=None, y=None, dt=M.BF16, acc=0, ws=None, nws=256):
    return lib.ep_expert_wgrad_bf16(C.byref(r or rows()), n, k, x or p(), dy or p(), b or p(), y or p(), dt, acc,
                                    ws or p(), nws, None)


def gemm4(lib, r=None, n=256, k=256, fmt=0, x=None, w=None, sc=None, b=None, y=None, dt=M.BF16, ws=None, nws=256):
    return lib.ep_expert_gemm_w4(C.byref(r or rows()), n, k, fmt, x or p(), w or p(), sc or p(), b or p(), y or p(), dt,
                                 ws or p(), nws, None)


def swiglu(lib, r=None, inner=256, gu=None, b=None, h=None, ws=None, nws=256):
    return lib.ep_swiglu(C.byref(r or rows()), inner, gu or p(), b or p(), h or p(), ws or p(), nws, None)


@pytest.mark.parametrize("i", range(len(BAD_ROWS)))
def test_bad_rows(lib, i):
    r, code = BAD_ROWS[i]
    for call in (gemm, wgrad, gemm4, swiglu):
        assert call(lib, r=r) == code, call.__name__
    info = B.moedisp_bf16_plan_info()
    assert lib.ep_bf16_plan_query(C.byref(r), 256, 256, C.byref(info), C.sizeof(info)) == code


@pytest.mark.parametrize("call", [gemm, wgrad, gemm4])
def test_sizes(lib, call):
    for n in (0, -8):
        assert call(lib, n=n) == B.ERR_INVALID_ARG
    for k in (0, -128):
        assert call(lib, k=k) == B.ERR_INVALID_ARG
    assert call(lib, n=(1 << 20) + 16) == B.ERR_UNSUPPORTED
    assert call(lib, k=65536 + 128) == B.ERR_UNSUPPORTED
    assert call(lib, n=260) == B.ERR_UNSUPPORTED
    assert call(lib, k=260) == B.ERR_UNSUPPORTED
    assert call(lib, dt=M.FP8_E4M3) == B.ERR_UNSUPPORTED
    assert call(lib, ws=p(64)) == B.ERR_MISALIGNED
    assert call(lib, nws=255) == B.ERR_WORKSPACE_TOO_SMALL
    assert call(lib, b=p(2)) == B.ERR_MISALIGNED
    for name in ("x", "y"):
        assert call(lib, **{name: p(8)}) == B.ERR_MISALIGNED
    # any hint is taken as one
    assert call(lib, r=rows(expected=2 ** 31 - 1), nws=255) == B.ERR_WORKSPACE_TOO_SMALL


def test_rules_of_their_own(lib):
    assert gemm(lib, lay=2) == B.ERR_UNSUPPORTED and gemm(lib, w=p(8)) == B.ERR_MISALIGNED
    assert wgrad(lib, acc=2, dt=M.FP32) == B.ERR_INVALID_ARG and wgrad(lib, acc=1) == B.ERR_UNSUPPORTED
    assert wgrad(lib, dy=p(8)) == B.ERR_MISALIGNED
    assert gemm4(lib, fmt=2) == B.ERR_UNSUPPORTED and gemm4(lib, n=264) == B.ERR_UNSUPPORTED
    assert gemm4(lib, k=192) == B.ERR_UNSUPPORTED
    assert gemm4(lib, w=p(8)) == B.ERR_MISALIGNED and gemm4(lib, sc=p(2)) == B.ERR_MISALIGNED
    # launches of more tiles than a grid holds
    big = rows(E=4096, R=(1 << 30) - 1)
    assert gemm(lib, r=big, n=1 << 20) == B.ERR_UNSUPPORTED and gemm4(lib, r=big, n=1 << 20) == B.ERR_UNSUPPORTED
    assert wgrad(lib, r=rows(E=4096), n=1 << 20, k=65536) == B.ERR_UNSUPPORTED
    for inner, code in ((0, B.ERR_INVALID_ARG), (192, B.ERR_UNSUPPORTED), (65536 + 128, B.ERR_UNSUPPORTED)):
        assert swiglu(lib, inner=inner) == code
    for name in ("gu", "h"):
        assert swiglu(lib, **{name: p(8)}) == B.ERR_MISALIGNED


def test_null_pointers(lib):
    r = C.byref(rows())
    for i in range(4):
        a = [p()] * 4
        a[i] = NULL
        assert lib.ep_expert_gemm_bf16(r, 256, 256, 0, *a, M.BF16, p(), 256, None) == B.ERR_INVALID_ARG, i
        assert lib.ep_expert_wgrad_bf16(r, 256, 256, *a, M.BF16, 0, p(), 256, None) == B.ERR_INVALID_ARG, i
    for i in range(5):
        a = [p()] * 5
        a[i] = NULL
        assert lib.ep_expert_gemm_w4(r, 256, 256, 0, *a, M.BF16, p(), 256, None) == B.ERR_INVALID_ARG, i
    for i in range(3):
        a = [p()] * 3
        a[i] = NULL
        assert lib.ep_swiglu(r, 256, *a, p(), 256, None) == B.ERR_INVALID_ARG, i
    a = [p()] * 4
    assert lib.ep_expert_gemm_bf16(None, 256, 256, 0, *a, M.BF16, p(), 256, None) == B.ERR_INVALID_ARG
    assert lib.ep_expert_gemm_bf16(r, 256, 256, 0, *a, M.BF16, None, 256, None) == B.ERR_INVALID_ARG


def router(**kw):
    d = dict(num_tokens=16, num_experts=64, topk=4, score=0, logits_dtype=M.FP32, groups=1, topk_groups=1, group_best=2,
             normalise=True, scale=1.0)
    d.update(kw)
    return M.moedisp_router.make(**d)


BAD_ROUTERS = [
    (dict(num_tokens=-1), B.ERR_INVALID_ARG), (dict(num_experts=0), B.ERR_INVALID_ARG), (dict(topk=0), B.ERR_INVALID_ARG),
    (dict(topk=65), B.ERR_INVALID_ARG), (dict(topk=33), B.ERR_UNSUPPORTED),
    (dict(num_experts=4104, groups=1), B.ERR_UNSUPPORTED), (dict(score=2), B.ERR_UNSUPPORTED),
    (dict(logits_dtype=M.FP8_E4M3), B.ERR_UNSUPPORTED), (dict(groups=0), B.ERR_INVALID_ARG),
    (dict(groups=3), B.ERR_INVALID_ARG), (dict(num_experts=128, groups=128), B.ERR_UNSUPPORTED),
    (dict(topk_groups=0), B.ERR_INVALID_ARG), (dict(groups=4, topk_groups=5), B.ERR_INVALID_ARG),
    (dict(group_best=0), B.ERR_INVALID_ARG), (dict(group_best=3), B.ERR_INVALID_ARG),
    (dict(scale=math.inf), B.ERR_INVALID_ARG), (dict(scale=math.nan), B.ERR_INVALID_ARG),
    (dict(num_tokens=1 << 28), B.ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("i", range(len(BAD_ROUTERS)))
def test_bad_routers(lib, i):
    kw, code = BAD_ROUTERS[i]
    r = router(**kw)
    assert lib.ep_router_topk(C.byref(r), p(), p(), p(), p(), p(), None) == code
    assert lib.ep_router_topk_backward(C.byref(r), p(), p(), p(), p(), p(), 256, None) == code
    info = B.moedisp_router_plan_info()
    assert lib.ep_router_plan_query(C.byref(r), C.byref(info), C.sizeof(info)) == code and info.struct_bytes == 0


def test_router_pointers(lib):
    r = router()
    r.normalise = 2
    assert lib.ep_router_topk(C.byref(r), p(), None, None, p(), p(), None) == B.ERR_INVALID_ARG
    r = C.byref(router())
    assert lib.ep_router_topk(None, p(), None, None, p(), p(), None) == B.ERR_INVALID_ARG
    for i in (0, 3, 4):
        a = [p(), NULL, NULL, p(), p()]
        a[i] = NULL
        assert lib.ep_router_topk(r, *a, None) == B.ERR_INVALID_ARG, i
    for i, off in ((0, 8), (1, 2), (3, 2), (4, 2)):
        a = [p()] * 5
        a[i] = p(off)
        assert lib.ep_router_topk(r, *a, None) == B.ERR_MISALIGNED, i
    for i in range(4):
        a = [p()] * 4
        a[i] = NULL
        assert lib.ep_router_topk_backward(r, *a, p(), 256, None) == B.ERR_INVALID_ARG, i
    for i, off in ((0, 8), (1, 2), (2, 2), (3, 8)):
        a = [p()] * 4
        a[i] = p(off)
        assert lib.ep_router_topk_backward(r, *a, p(), 256, None) == B.ERR_MISALIGNED, i
    assert lib.ep_router_topk_backward(r, p(), p(), p(), p(), None, 256, None) == B.ERR_INVALID_ARG
    assert lib.ep_router_topk_backward(r, p(), p(), p(), p(), p(), 255, None) == B.ERR_WORKSPACE_TOO_SMALL


def test_plans(lib):
    for E, lanes, per in ((1, 16, 4), (64, 16, 4), (65, 16, 8), (256, 64, 4), (257, 64, 8), (1024, 64, 16), (4096, 64, 64)):
        info = M.ep_router_plan_query(M.moedisp_router.make(8, E, 1))
        assert (info["lanes"], info["per_lane"]) == (lanes, per)
        assert info["lanes"] * info["per_lane"] >= E
    assert M.ep_router_plan_query(M.moedisp_router.make(100000, 256, 1))["lanes"] == 16
    for E in (1, 8, 64, 4096):
        for n in (16, 264, 4096, 1 << 20):
            for rows_ in (1, 16, 64, 128, 1000, 2 ** 30, 2 ** 31 - 1):
                i = M.ep_bf16_plan_query(M.moedisp_rows.contiguous(E, 1 << 20, rows_), n, 512)
                assert i["product_rows"] in (32, 64, 96, 128, 160, 256) and i["int4_rows"] in (16, 32, 64, 96, 160)
    assert M.ep_bf16_plan_query(M.moedisp_rows.contiguous(8, 64), 4096, 4096)["wgrad_cols"] == 256
    assert M.ep_bf16_plan_query(M.moedisp_rows.contiguous(8, 64), 512, 512)["wgrad_cols"] == 128


def test_binding_rejects_bad_tensors():
    """Wrong types, sizes and strides raise before the call; so do tensors that
    are not on a GPU."""
    r = M.moedisp_rows.contiguous(2, 4)
    bounds, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    x, w, y = (torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 64, dtype=torch.bfloat16),
               torch.zeros(4, 64, dtype=torch.bfloat16))

    def fails(text, f, *a):
        with pytest.raises(M.MoeDispError, match=text):
            f(*a)

    fails("x has dtype", M.ep_expert_gemm_bf16, r, 64, 64, 0, x.float(), w, bounds, y, M.BF16, ws)
    fails("w holds", M.ep_expert_gemm_bf16, r, 64, 64, 0, x, w[:1], bounds, y, M.BF16, ws)
    fails("contiguous", M.ep_expert_gemm_bf16, r, 64, 64, 0, x, w.transpose(1, 2), bounds, y, M.BF16, ws)
    fails("y has dtype", M.ep_expert_gemm_bf16, r, 64, 64, 0, x, w, bounds, y, M.FP32, ws)
    fails("y overlaps x", M.ep_expert_gemm_bf16, r, 64, 64, 0, x, w, bounds, x, M.BF16, ws)
    fails("expected a GPU tensor", M.ep_expert_gemm_bf16, r, 64, 64, 0, x, w, bounds, y, M.BF16, ws)
    fails("dw has dtype", M.ep_expert_wgrad_bf16, r, 64, 64, x, y, bounds, w, M.FP32, False, ws)
    fails("w_scales has dtype", M.ep_expert_gemm_w4, r, 64, 64, M.W4_E2M1, x, w.view(torch.uint8), w, bounds, y, M.BF16, ws)
    fails("h holds", M.ep_swiglu, r, 128, torch.zeros(4, 256, dtype=torch.bfloat16), bounds, y, ws)
    rt = M.moedisp_router.make(4, 8, 2)
    z, idx, wt = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    fails("logits has dtype", M.ep_router_topk, rt, z.bfloat16(), None, None, idx, wt)
    fails("topk_idx has dtype", M.ep_router_topk, rt, z, None, None, idx.long(), wt)
    fails("live has dtype", M.ep_router_topk, rt, z, None, torch.ones(4), idx, wt)
    fails("bias holds", M.ep_router_topk, rt, z, torch.zeros(7), None, idx, wt)
    fails("d_logits overlaps logits", M.ep_router_topk_backward, rt, z, idx, wt, z, ws)
    fails("expected a GPU tensor", M.ep_router_topk, rt, z, None, None, idx, wt)

