"""CPU checks of the 8-bit product: layout, argument order of the binding, refusals before any launch."""
import ctypes

import pytest
import torch

import int4_expert_ffn_top_b200 as M
from int4_expert_ffn_top_b200 import _lib
from int4_expert_ffn_top_b200 import build as B
from test_binding_checks import cu, f32, i32, rec  # noqa: F401  (fixture)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


def test_row_bytes(lib):
    assert [lib.moe_i8_row_bytes(n) for n in (0, -3, 1, 16, 17, 65536, 65537)] == [0, 0, 16, 16, 32, 65536, 0]


def test_rows_are_padded_with_zeros_once():
    codes = torch.randint(-128, 128, (5, 19), dtype=torch.int8)
    d = M.DeviceLinear8(codes, torch.ones(5))
    assert d.codes.shape == (5, 32) and torch.equal(d.codes[:, :19], codes) and (d.codes[:, 19:] == 0).all()
    assert (d.struct.ld, d.struct.out_dim, d.struct.in_dim, d.struct.bias) == (32, 5, 19, None)
    whole = torch.zeros((4, 32), dtype=torch.int8)
    assert M.DeviceLinear8(whole, torch.ones(4)).codes.data_ptr() == whole.data_ptr()
    turned = torch.randint(-128, 128, (32, 16), dtype=torch.int8).T
    assert torch.equal(M.DeviceLinear8(turned, torch.ones(16)).codes, turned)
    for bad in (lambda: M.DeviceLinear8(codes.float(), torch.ones(5)), lambda: M.DeviceLinear8(codes, torch.ones(4)),
                lambda: M.DeviceLinear8(codes, torch.ones(5), torch.ones(5).double()),
                lambda: M.DeviceLinear8(codes[:0], torch.ones(0))):
        with pytest.raises(ValueError):
            bad()


def test_library_refuses_bad_calls(lib):
    bad, uns = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED
    A = 1 << 20

    def quant(x=A, kind=0, T=1, H=64, eps=-1.0, q=A, ld=64, scale=A):
        return lib.moe_quant_i8(x, kind, T, H, eps, q, ld, scale, None)

    assert quant(T=0) == _lib.MOE_OK and quant(T=0, x=None, q=None, scale=None) == _lib.MOE_OK
    for kw in (dict(kind=2), dict(eps=float("nan")), dict(ld=48), dict(ld=72), dict(x=None), dict(q=None),
               dict(q=A + 8), dict(scale=None)):
        assert quant(**kw) == bad, kw
    for kw in (dict(T=-1), dict(T=_lib.MOE_MAX_TOKENS + 1), dict(H=0), dict(H=65537, ld=65552)):
        assert quant(**kw) == uns, kw

    def product(codes=A, ld=64, scale=A, n=8, k=64, q=A, ldq=64, qs=A, T=1, out=A, mode=0):
        W = _lib.moe_linear8(codes, ld, scale, None, n, k)
        return lib.moe_linear_i8(ctypes.byref(W), q, ldq, qs, T, out, mode, None, None)

    assert product(T=0) == _lib.MOE_OK and product(T=0, q=None, qs=None, out=None) == _lib.MOE_OK
    assert lib.moe_linear_i8(None, A, 64, A, 1, A, 0, None, None) == bad
    for kw in (dict(codes=None), dict(codes=A + 4), dict(ld=48), dict(ld=70), dict(scale=None), dict(q=None),
               dict(q=A + 1), dict(ldq=32), dict(ldq=65), dict(qs=None), dict(out=None), dict(mode=3), dict(mode=-1)):
        assert product(**kw) == bad, kw
    for kw in (dict(T=-1), dict(T=_lib.MOE_MAX_TOKENS + 1), dict(n=0), dict(n=1048577), dict(k=0),
               dict(k=65537, ld=65552, ldq=65552)):
        assert product(**kw) == uns, kw


def test_library_refuses_addresses_that_no_element_can_have(lib):
    bad, A = _lib.MOE_ERR_INVALID_ARG, 1 << 20
    for kind, x, scale in ((0, A + 2, A), (0, A + 1, A), (1, A + 1, A), (0, A, A + 2), (1, A + 2, A + 1)):
        assert lib.moe_quant_i8(x, kind, 1, 64, -1.0, A, 64, scale, None) == bad
    for scale, bias, qs, out, mode, err in ((A + 2, None, A, A, 0, None), (A, A + 1, A, A, 0, None), (A, None, A + 2, A, 0, None),
                                            (A, None, A, A + 2, 0, None), (A, None, A, A + 2, 2, None),
                                            (A, None, A, A + 1, 1, None), (A, None, A, A, 0, A + 2)):
        W = _lib.moe_linear8(A, 64, scale, bias, 8, 64)
        assert lib.moe_linear_i8(ctypes.byref(W), A, 64, qs, 1, out, mode, err, None) == bad


def test_product_takes_no_read_only_loads():
    """What the kernel ahead may be writing when the product starts is not read through the read-only path, whose loads a
    compiler may move above the wait for that kernel."""
    import os
    import re
    with open(os.path.join(os.path.dirname(B.__file__), "csrc", "linear8.cuh")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "griddepcontrol.wait" in code
    assert not re.findall(r"__ldg|ldg_stream|global\.nc|__restrict__", code)


class FakeLinear:
    def __init__(self, n, k):
        self.struct = _lib.moe_linear8(1 << 20, (k + 15) // 16 * 16, 1 << 20, None, n, k)
        self.device = torch.device("cuda", 0)


def i8(*shape):
    return cu(torch.zeros(shape, dtype=torch.int8))


def test_binding_order_and_checks(rec):  # noqa: F811
    x, q, s = f32(5, 60), i8(5, 64), f32(5)
    M.moe_quant_i8(x, q, s, stream=0)
    assert rec.calls[-1] == ("moe_quant_i8", (x.data_ptr(), 0, 5, 60, -1.0, q.data_ptr(), 64, s.data_ptr(), 0))
    xb = cu(torch.zeros((5, 60), dtype=torch.bfloat16))
    M.moe_quant_i8(xb, q, s, eps=1e-5, stream=0)
    assert rec.calls[-1][1][1:5] == (1, 5, 60, 1e-5)
    lin, out = FakeLinear(7, 60), f32(5, 7)
    M.moe_linear_i8(lin, q, s, out, M.OUT_ADD_F32, stream=0)
    assert rec.calls[-1][1][1:] == (q.data_ptr(), 64, s.data_ptr(), 5, out.data_ptr(), 2, None, 0)
    err = i32(1)
    out16 = cu(torch.zeros((5, 7), dtype=torch.int16))
    M.moe_linear_i8(lin, q, s, out16, M.OUT_BF16, err_word=err, stream=0)
    assert rec.calls[-1][1][-4:] == (out16.data_ptr(), 1, err.data_ptr(), 0)
    n = len(rec.calls)
    for call in (lambda: M.moe_quant_i8(x, i8(5, 62), s), lambda: M.moe_quant_i8(x, i8(5, 48), s),
                 lambda: M.moe_quant_i8(x, i8(4, 64), s), lambda: M.moe_quant_i8(x, q, f32(4)),
                 lambda: M.moe_quant_i8(x.double(), q, s), lambda: M.moe_quant_i8(x, q, s, eps=-1.0),
                 lambda: M.moe_quant_i8(x, q, s, eps=float("nan")), lambda: M.moe_quant_i8(x[0], q, s),
                 lambda: M.moe_quant_i8(torch.zeros(5, 60), q, s), lambda: M.moe_quant_i8(f32(60, 5).T, q, s),
                 lambda: M.moe_linear_i8(FakeLinear(7, 65), q, s, out, 0), lambda: M.moe_linear_i8(lin, q, f32(4), out, 0),
                 lambda: M.moe_linear_i8(lin, q, s, f32(34), 0), lambda: M.moe_linear_i8(lin, q, s, out16, 0),
                 lambda: M.moe_linear_i8(lin, i8(5, 128)[:, :64], s, out, 0)):
        with pytest.raises((ValueError, TypeError)):
            call()
    assert len(rec.calls) == n


def test_extension_belongs_to_this_torch(lib, monkeypatch):
    """Built for another torch it is built again, and is not used meanwhile."""
    assert not B.binding_stale() and _lib.binding().built_for == B.binding_tag()
    monkeypatch.setattr(torch, "__version__", "2.1.0")
    assert B.binding_stale()
    monkeypatch.setattr(_lib, "_fast", None)
    with pytest.raises(RuntimeError, match="this is torch 2.1.0"):
        _lib.binding()


def test_quick_way_takes_nothing_it_has_not_checked(lib):
    """The extension answers None, without a call, to anything but tensors on the current CUDA device."""
    b = _lib.binding()
    x, q, s = torch.zeros((2, 64)), torch.zeros((2, 64), dtype=torch.int8), torch.zeros(2)
    W = ctypes.addressof(_lib.moe_linear8(None, 64, None, None, 8, 64))
    assert b.quant(x, q, s, None) is None and b.quant(x, q, s, float("nan")) is None and b.quant(x, q, s, "1") is None
    assert b.quant(x, q, s) is None and b.quant(None, None, None, None) is None
    assert b.linear(W, 0, q, s, x, 0, None) is None and b.linear(0, 0, q, s, x, 0, None) is None
    assert b.linear(W, None, q, s, x, 0, None) is None and b.linear("w", 0, q, s, x, 0, None) is None
    L = _lib.moe_layer()
    A = ctypes.addressof(L)
    assert b.layer(A, x, None, 1e-6, 2, None, None, q, s, x, 0, q, None) is None
    assert b.layer(A, None, x, 1e-6, 99, None, None, q, s, x, 0, q, None) is None
    assert b.layer(A, None, x, "eps", 2, None, None, q, s, x, 0, q, None) is None
