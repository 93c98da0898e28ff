"""Argument checks of the experts' products, the gated activation and the
balance loss (no GPU needed): every call below is rejected on the host, with
the documented code, before anything touches a device."""
import ctypes as C
import math
import os

import pytest
import torch

import combine_ep_get_dispatch_amd as M
from combine_ep_get_dispatch_amd import binding as B


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from combine_ep_get_dispatch_amd import build
        build.build()
    return M.load()


FAKE = 0x10000  # never dereferenced


def p(off=0):
    return C.c_void_p(FAKE + off)


def rows(E=8, R=64, **kw):
    return M.moedisp_rows(E, R, kw.get("stride", 0), kw.get("cap", 0), kw.get("base", 0), kw.get("expected", 0))


BAD_ROWS = [
    (rows(E=0), B.ERR_INVALID_ARG), (rows(R=-1), B.ERR_INVALID_ARG), (rows(expected=-1), B.ERR_INVALID_ARG),
    (rows(E=4097), B.ERR_UNSUPPORTED), (rows(R=1 << 30), B.ERR_UNSUPPORTED),
    (rows(cap=3), B.ERR_INVALID_ARG), (rows(base=1), B.ERR_INVALID_ARG),           # contiguous rows have neither
    (rows(stride=8, cap=9), B.ERR_INVALID_ARG), (rows(stride=8, cap=4, base=5), B.ERR_INVALID_ARG),
    (rows(stride=8, cap=-1), B.ERR_INVALID_ARG), (rows(stride=8, cap=4, base=-1), B.ERR_INVALID_ARG),
    (rows(stride=-8), B.ERR_INVALID_ARG), (rows(R=65, stride=8, cap=8), B.ERR_INVALID_ARG),  # R != E * stride
]


def gemm(lib, r=None, n=256, k=256, fmt=0, x=None, xs=None, w=None, wsc=None, b=None, y=None, dt=M.BF16, ws=None,
         nws=256):
    return lib.ep_expert_gemm(C.byref(r or rows()), n, k, fmt, x or p(), xs or p(), w or p(), wsc or p(), b or p(),
                              y or p(), dt, ws or p(), nws, None)


def wgrad(lib, r=None, n=256, k=256, fmt=0, x=None, xs=None, dy=None, b=None, dw=None, dt=M.BF16, acc=0, ws=None,
          nws=256):
    return lib.ep_expert_wgrad(C.byref(r or rows()), n, k, fmt, x or p(), xs or p(), dy or p(), b or p(), dw or p(),
                               dt, acc, ws or p(), nws, None)


def swiglu(lib, r=None, inner=256, fmt=0, gu=None, b=None, h=None, hs=None, ws=None, nws=256):
    return lib.ep_swiglu_quant(C.byref(r or rows()), inner, fmt, gu or p(), b or p(), h or p(), hs or p(),
                               ws or p(), nws, None)


NULL = C.c_void_p(None)


def swiglu_backward(lib, r=None, inner=256, fmt=0, gu=None, dh=None, b=None, dgu=p(), q=p(), qs=p(), ws=None,
                    nws=256):
    return lib.ep_swiglu_backward(C.byref(r or rows()), inner, fmt, gu or p(), dh or p(), b or p(), dgu, q, qs,
                                  ws or p(), nws, None)


@pytest.mark.parametrize("i", range(len(BAD_ROWS)))
def test_bad_rows(lib, i):
    r, code = BAD_ROWS[i]
    for call in (gemm, wgrad, swiglu, swiglu_backward):
        assert call(lib, r=r) == code, call.__name__


@pytest.mark.parametrize("call", [gemm, wgrad])
def test_product_sizes(lib, call):
    for n in (0, -8):
        assert call(lib, n=n) == B.ERR_INVALID_ARG
    for k in (0, -128):
        assert call(lib, k=k) == B.ERR_INVALID_ARG
    assert call(lib, n=12) == B.ERR_UNSUPPORTED                 # rows of whole 16-byte units
    assert call(lib, k=192) == B.ERR_UNSUPPORTED                # whole scale blocks
    assert call(lib, k=65536 + 128) == B.ERR_UNSUPPORTED
    assert call(lib, n=(1 << 20) + 8) == B.ERR_UNSUPPORTED
    assert call(lib, fmt=2) == B.ERR_UNSUPPORTED
    assert call(lib, dt=M.FP8_E4M3) == B.ERR_UNSUPPORTED
    assert call(lib, ws=p(64)) == B.ERR_MISALIGNED
    assert call(lib, nws=255) == B.ERR_WORKSPACE_TOO_SMALL
    assert call(lib, b=p(2)) == B.ERR_MISALIGNED
    assert call(lib, x=p(8)) == B.ERR_MISALIGNED
    assert call(lib, xs=p(2)) == B.ERR_MISALIGNED
    # any hint is taken as one
    assert call(lib, r=rows(expected=2 ** 31 - 1), nws=255) == B.ERR_WORKSPACE_TOO_SMALL
    # a launch of more tiles than a grid holds
    assert gemm(lib, r=rows(E=4096, R=(1 << 30) - 1), n=1 << 20) == B.ERR_UNSUPPORTED
    assert wgrad(lib, r=rows(E=4096), n=1 << 20, k=65536) == B.ERR_UNSUPPORTED


def test_product_pointers(lib):
    for name in ("w", "y"):
        assert gemm(lib, **{name: p(8)}) == B.ERR_MISALIGNED
    assert gemm(lib, wsc=p(1)) == B.ERR_MISALIGNED
    for name in ("dy", "dw"):
        assert wgrad(lib, **{name: p(8)}) == B.ERR_MISALIGNED
    r = rows()
    args = [p(), p(), p(), p(), p(), p()]
    for i in range(6):
        a = list(args)
        a[i] = NULL
        assert lib.ep_expert_gemm(C.byref(r), 256, 256, 0, *a, M.BF16, p(), 256, None) == B.ERR_INVALID_ARG, i
    for i in range(5):
        a = list(args[:5])
        a[i] = NULL
        assert lib.ep_expert_wgrad(C.byref(r), 256, 256, 0, *a, M.BF16, 0, p(), 256, None) == B.ERR_INVALID_ARG, i
    assert lib.ep_expert_gemm(None, 256, 256, 0, *args, M.BF16, p(), 256, None) == B.ERR_INVALID_ARG
    assert lib.ep_expert_gemm(C.byref(r), 256, 256, 0, *args, M.BF16, None, 256, None) == B.ERR_INVALID_ARG
    assert wgrad(lib, acc=2, dt=M.FP32) == B.ERR_INVALID_ARG
    assert wgrad(lib, acc=1, dt=M.BF16) == B.ERR_UNSUPPORTED    # sums of gradients are kept in binary32


def test_swiglu_arguments(lib):
    for call in (swiglu, swiglu_backward):
        assert call(lib, inner=0) == B.ERR_INVALID_ARG
        assert call(lib, inner=192) == B.ERR_UNSUPPORTED
        assert call(lib, inner=65536 + 128) == B.ERR_UNSUPPORTED
        assert call(lib, fmt=-1) == B.ERR_UNSUPPORTED
        assert call(lib, gu=p(8)) == B.ERR_MISALIGNED
        assert call(lib, ws=p(128)) == B.ERR_MISALIGNED
        assert call(lib, nws=0) == B.ERR_WORKSPACE_TOO_SMALL
    assert swiglu(lib, hs=p(2)) == B.ERR_MISALIGNED
    assert swiglu(lib, h=p(4)) == B.ERR_MISALIGNED
    assert swiglu_backward(lib, dgu=p(8)) == B.ERR_MISALIGNED
    assert swiglu_backward(lib, qs=p(2)) == B.ERR_MISALIGNED
    assert swiglu_backward(lib, q=NULL) == B.ERR_INVALID_ARG             # codes without scales, or the reverse
    assert swiglu_backward(lib, qs=NULL) == B.ERR_INVALID_ARG
    assert swiglu_backward(lib, dgu=NULL, q=NULL, qs=NULL) == B.ERR_INVALID_ARG
    assert swiglu_backward(lib, dh=p(8)) == B.ERR_MISALIGNED


def balance(S=2, L=8, E=16, k=2, score=0, dt=M.FP32, coef=1.0):
    return M.moedisp_balance.make(S, L, E, k, score, dt, coef)


def test_balance_arguments(lib):
    def fwd(b, z=None, idx=None, loss=None, c=None, t=None, ws=None, nws=1 << 30):
        return lib.ep_balance_loss(C.byref(b), z or p(), idx or p(), loss or p(), c or p(), t or p(), ws or p(), nws,
                                   None)

    def bwd(b, z=None, idx=None, c=None, t=None, d=None, dz=None):
        return lib.ep_balance_loss_backward(C.byref(b), z or p(), idx or p(), c or p(), t or p(), d or p(),
                                            dz or p(), None)

    bad = [(balance(S=-1), B.ERR_INVALID_ARG), (balance(L=-1), B.ERR_INVALID_ARG), (balance(E=0), B.ERR_INVALID_ARG),
           (balance(k=0), B.ERR_INVALID_ARG), (balance(k=17), B.ERR_INVALID_ARG),
           (balance(coef=math.inf), B.ERR_INVALID_ARG), (balance(coef=math.nan), B.ERR_INVALID_ARG),
           (balance(E=4097), B.ERR_UNSUPPORTED), (balance(E=64, k=33), B.ERR_UNSUPPORTED),
           (balance(score=2), B.ERR_UNSUPPORTED), (balance(dt=M.FP8_E4M3), B.ERR_UNSUPPORTED),
           (balance(S=1 << 15, L=1 << 15, k=1), B.ERR_UNSUPPORTED)]
    for b, code in bad:
        assert fwd(b) == code and bwd(b) == code, b
        assert M.ep_balance_workspace_bytes(b) == 0
    b = balance()
    need = M.ep_balance_workspace_bytes(b)
    assert need >= 256 and need % 256 == 0
    assert fwd(b, nws=need - 1) == B.ERR_WORKSPACE_TOO_SMALL
    assert fwd(b, ws=p(64)) == B.ERR_MISALIGNED
    for name in ("z", "idx", "loss", "c", "t"):
        assert fwd(b, **{name: p(2)}) == B.ERR_MISALIGNED, name
    for name in ("z", "idx", "c", "t", "d", "dz"):
        assert bwd(b, **{name: p(2)}) == B.ERR_MISALIGNED, name
    assert lib.ep_balance_loss(C.byref(b), p(), p(), None, p(), p(), p(), need, None) == B.ERR_INVALID_ARG
    assert lib.ep_balance_loss(None, p(), p(), p(), p(), p(), p(), need, None) == B.ERR_INVALID_ARG
    assert lib.ep_balance_loss_backward(C.byref(b), p(), p(), p(), p(), None, p(), None) == B.ERR_INVALID_ARG
    # more sequences than one launch takes: refused before the first launch
    assert fwd(balance(S=1 << 22, L=1, E=64, k=1), nws=1 << 40) == B.ERR_UNSUPPORTED
    assert bwd(balance(S=1 << 25, L=1, E=8, k=1)) == B.ERR_UNSUPPORTED
    # the workspace does not overflow at the largest batch and expert count
    assert M.ep_balance_workspace_bytes(balance(S=(1 << 30) - 1, L=1, E=4096, k=1)) > (1 << 42)


def t(*shape, dt=torch.uint8):
    return torch.zeros(*shape, dtype=dt)


def test_binding_checks_tensors():
    """Sizes, types, overlap and placement are checked before the C call."""
    r = M.moedisp_rows.contiguous(4, 16)
    ok = dict(x=t(16, 128), x_scales=t(16, 1, dt=torch.float32), w=t(4, 8, 128), w_scales=t(4, 1, 1, dt=torch.float32),
              row_bounds=t(5, dt=torch.int32), y=t(16, 8, dt=torch.bfloat16), ws=t(256))

    def call(fmt=M.SCALE_FP32, out=M.BF16, **kw):
        a = dict(ok, **kw)
        M.ep_expert_gemm(r, 8, 128, fmt, a["x"], a["x_scales"], a["w"], a["w_scales"], a["row_bounds"], a["y"], out,
                         a["ws"])

    with pytest.raises(M.MoeDispError, match="expected a GPU tensor"):
        call()
    for name, bad, text in (("x", t(15, 128), "holds"), ("x", t(16, 128, dt=torch.int32), "dtype"),
                            ("x_scales", t(16, 1), "dtype"), ("w", t(4, 8, 127), "holds"),
                            ("w", t(8, 4, 128).transpose(0, 1), "contiguous"), ("row_bounds", t(4, dt=torch.int32), "holds"),
                            ("row_bounds", t(5, dt=torch.int64), "dtype"), ("y", t(16, 8), "holds"),
                            ("w_scales", None, "required")):
        with pytest.raises(M.MoeDispError, match=text):
            call(**{name: bad})
    with pytest.raises(M.MoeDispError, match="dtype"):
        call(fmt=M.SCALE_UE8M0)
    with pytest.raises(M.MoeDispError, match="dtype"):
        call(out=M.FP32)
    big = t(16, 128)
    with pytest.raises(M.MoeDispError, match="overlaps"):
        call(x=big, y=big.view(-1)[:256].view(torch.bfloat16))
    with pytest.raises(M.MoeDispError, match="31 bits"):
        M.moedisp_rows.padded(4096, 1 << 20)
