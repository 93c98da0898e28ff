"""The binding's argument checks in C++ and in Python say the same (no GPU
needed for what is refused; with one, that both find the same addresses,
GPU and stream)."""
import os
import sys

import pytest
import torch

from combine_ep_get_dispatch_amd import binding as B
from combine_ep_get_dispatch_amd.build import CHECKS

PyArgs = type("PyArgs", (B._PyChecks,), {n: B._Args.__dict__[n] for n in ("fail", "need", "done", "resolve")})
BOTH = [B._Args, PyArgs]


@pytest.mark.skipif(not os.path.exists(CHECKS), reason="_checks.so is not built; the checks run in Python")
def test_the_native_checks_are_in_use():
    from combine_ep_get_dispatch_amd import _checks
    assert issubclass(B._Args, _checks.Checks)


def outcome(cls, calls, stream=None, device=True):
    """What a series of arg() calls and on_device() give, or the error's text."""
    A = cls("some_call")
    try:
        got = [A.arg(*a, **kw) for a, kw in calls]
        return got, A.on_device(stream) if device else None
    except (B.MoeDispError, RuntimeError) as e:
        return str(e)


x = torch.zeros(8, 16, dtype=torch.bfloat16)
i = torch.zeros(9, dtype=torch.int32)
REFUSED = [
    ([(("x", x.float(), B._ROWS_BF16, 1), {})], "x has dtype float32"),
    ([(("x", x, B._ROWS_BF16, 257), {})], "x holds 256 bytes"),
    ([(("x", x.t(), B._ROWS_BF16, 1), {})], "x must be contiguous"),
    ([(("x", None, B._ROWS_BF16, 1), {})], "x is required"),
    ([(("x", [1], B._ROWS_BF16, 1), {})], "x must be a torch.Tensor"),
    ([(("x", x, B._ROWS_BF16, 256), {}), (("y", x[2:4], B._ROWS_BF16, 1), dict(written=True))], "y overlaps x"),
    ([(("y", x, None, 1), dict(written=True)), (("z", x, None, 1), dict(written=True))], "y overlaps z"),
    ([(("x", x, B._ROWS_BF16, 256), {}), (("i", i, B._INT32, 36), {})], "x is on cpu"),
    ([(("x", x.to_sparse(), B._ROWS_BF16, 1), {})], ""),
]


@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_refusals(case):
    calls, text = REFUSED[case]
    a, b = (outcome(c, calls) for c in BOTH)
    assert isinstance(a, str) and isinstance(b, str) and text in a
    assert a == b or not text


def test_addresses():
    par = torch.nn.Parameter(torch.zeros(4))
    calls = [(("x", x, B._ROWS_BF16, 256), {}), (("tail", x[3:], None, 32), dict(written=True)),
             (("none", None, B._F32, 8), dict(optional=True)), (("empty", None, B._F32, 0), {}),
             (("positional", i, B._INT32, 36, True, True), {}), (("par", par, B._F32, 16), {}),
             (("zero", torch.empty(0, 4), B._F32, 0), {})]
    a, b = (outcome(c, calls, device=False) for c in BOTH)
    assert a == b
    assert a[0][0] == x.data_ptr() and a[0][1] == x[3:].data_ptr() and a[0][2] is None


def test_no_reference_is_kept():
    before = sys.getrefcount(i), sys.getrefcount(B._INT32)
    for _ in range(100):
        A = B._Args("c")
        A.arg("i", i, B._INT32, 36)
        with pytest.raises(B.MoeDispError):
            A.arg("j", i, B._F32, 36)
        with pytest.raises(B.MoeDispError):
            A.on_device(None)
        del A
    assert (sys.getrefcount(i), sys.getrefcount(B._INT32)) == before


def test_misuse_raises():
    A = B._Args("c")
    for bad in (("x",), ("x", x, None, "many"), ("x", x, [torch.int32], 1)):
        with pytest.raises(TypeError):
            A.arg(*bad)
    with pytest.raises(TypeError):
        A.arg("x", x, None, 1, wrong=True)
    with pytest.raises(TypeError):
        for _ in range(40):
            A.arg("x", x, None, 1)


@pytest.mark.gpu
def test_on_a_gpu():
    g, o, j = x.cuda(), torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda"), i.cuda()
    calls = [(("g", g, B._ROWS_BF16, 256), {}), (("j", j, B._INT32, 36), {}), (("o", o, B._ROWS_BF16, 256), dict(written=True))]
    side = torch.cuda.Stream()
    for stream in (None, side):
        a, b = (outcome(c, calls, stream) for c in BOTH)
        assert a == b and a[1][0] == g.get_device()
        assert a[1][1] == (stream or torch.cuda.current_stream()).cuda_stream
    with torch.cuda.stream(side):
        a, b = (outcome(c, calls) for c in BOTH)
        assert a == b and a[1][1] == side.cuda_stream
    for more in ((("x", x, None, 1), {}), (("w", g[1:], None, 1), dict(written=True))):
        a, b = (outcome(c, calls + [more]) for c in BOTH)
        assert isinstance(a, str) and a == b
