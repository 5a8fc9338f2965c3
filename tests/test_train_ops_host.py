"""Host-side checks of the training operators' C ABI, without a GPU: bad
descriptions are refused before the device is touched, empty calls are no-ops,
workspace queries follow strides and types."""
import ctypes

import pytest
import torch

from group_limited_routed_gb300 import api

OK, INVALID, WORKSPACE = 0, 1, 3
P, I64, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t


@pytest.fixture(scope="module")
def lib():
    from group_limited_routed_gb300 import build
    build.build()
    return api.lib()


def desc(**kw):
    d = dict(rows=100, n_groups=4, N=64, K=128, dtype=0, out_dtype=0, x_ld=128, y_ld=64,
             w_stride_e=64 * 128, w_stride_n=128, w_stride_k=1)
    d.update(kw)
    return api._Grouped(*(d[n] for n, _ in api._Grouped._fields_))


BAD = [dict(rows=-1), dict(n_groups=0), dict(n_groups=1025), dict(N=0), dict(K=0), dict(dtype=2),
       dict(dtype=7), dict(out_dtype=1), dict(x_ld=127), dict(y_ld=63), dict(w_stride_k=2),
       dict(w_stride_n=127), dict(w_stride_e=-8), dict(w_stride_n=1, w_stride_k=63),
       dict(x_ld=1 << 39)]


@pytest.mark.parametrize("kw", BAD, ids=str)
def test_bad_grouped_descriptions(lib, kw):
    d = desc(**kw)
    r = ctypes.byref(d)
    assert lib.beam_moe_grouped_matmul_workspace_size(r, 0) == 0
    assert lib.beam_moe_grouped_matmul(r, None, None, None, None, None, 0, None) == INVALID
    assert lib.beam_moe_grouped_matmul_dx(r, None, None, None, None, None, 0, None) == INVALID
    assert lib.beam_moe_grouped_matmul_dw(r, None, None, None, 0, None, None, 0, None) == INVALID


def test_grouped_calls_without_rows_or_pointers(lib):
    d = desc(rows=0)
    r = ctypes.byref(d)
    assert lib.beam_moe_grouped_matmul(r, None, None, None, None, None, 0, None) == OK
    assert lib.beam_moe_grouped_matmul_dx(r, None, None, None, None, None, 0, None) == OK
    # the weight gradient still has to be written
    assert lib.beam_moe_grouped_matmul_dw(r, None, None, None, 0, None, None, 0, None) == INVALID
    f32 = desc(rows=0, out_dtype=2)
    assert lib.beam_moe_grouped_matmul_dw(ctypes.byref(f32), None, None, None, 1, P(256), P(256),
                                          256, None) == OK      # adds nothing
    d = desc()
    r = ctypes.byref(d)
    assert lib.beam_moe_grouped_matmul(r, None, None, None, None, P(256), 256, None) == INVALID
    # 16-bit sums are not added to; a misaligned workspace
    assert lib.beam_moe_grouped_matmul_dw(r, P(256), P(256), P(256), 1, P(256), P(256), 256,
                                          None) == INVALID
    assert lib.beam_moe_grouped_matmul(r, P(256), P(256), P(256), P(256), P(264), 256,
                                       None) == INVALID


def test_grouped_workspace_follows_alignment(lib):
    size = lambda **kw: lib.beam_moe_grouped_matmul_workspace_size(ctypes.byref(desc(**kw)), 0)
    assert size() == 256
    packed = lambda *dims: (2 * dims[0] * dims[1] * dims[2] + 255) // 256 * 256
    assert size(x_ld=129) == 256 + packed(1, 100, 128)
    assert size(K=127, x_ld=127, w_stride_n=127, w_stride_e=127 * 64) == \
        256 + packed(1, 100, 128) + packed(4, 64, 128)
    # a transposed view of aligned weights needs no copy
    assert size(w_stride_n=1, w_stride_k=64) == 256
    every = lib.beam_moe_grouped_matmul_workspace_size(ctypes.byref(desc()), 1)
    assert every == 256 + packed(1, 100, 128) + packed(1, 100, 64) + packed(4, 64, 128)
    # an operand that has to be copied does not fit in the status word's 256 bytes
    d = desc(x_ld=129)
    assert lib.beam_moe_grouped_matmul(ctypes.byref(d), P(256), P(256), P(256), P(256), P(256),
                                       256, None) == WORKSPACE


def test_gate_checks(lib):
    g = api._Gate(0, 64, 0, 64, 64)
    assert lib.beam_moe_swiglu(ctypes.byref(g), None, None, None, None, 64, None) == OK
    assert lib.beam_moe_swiglu_grad(ctypes.byref(g), None, 64, None, None, None, None, 64, None,
                                    64, None, None) == OK
    for bad in (api._Gate(-1, 64, 0, 64, 64), api._Gate(4, -1, 0, 64, 64),
                api._Gate(4, 64, 2, 64, 64), api._Gate(4, 64, 0, 63, 64),
                api._Gate(4, 64, 0, 64, 63)):
        assert lib.beam_moe_swiglu(ctypes.byref(bad), None, None, None, None, 64, None) == INVALID
        assert lib.beam_moe_swiglu_grad(ctypes.byref(bad), None, 64, None, None, None, None, 64,
                                        None, 64, None, None) == INVALID
    assert lib.beam_moe_swiglu(None, None, None, None, None, 64, None) == INVALID


def test_orthogonalize_checks(lib):
    def ortho(**kw):
        d = dict(batch=1, rows=8, cols=8, dtype=0, out_dtype=0, steps=5, a=3.4, b=-4.8, c=2.0,
                 eps=1e-7, stride_batch=64, stride_row=8, stride_col=1)
        d.update(kw)
        o = api._Ortho(*(d[n] for n, _ in api._Ortho._fields_))
        return lib.beam_moe_orthogonalize(ctypes.byref(o), None, None, None, 0, None)
    nan, inf = float("nan"), float("inf")
    for kw in (dict(batch=-1), dict(batch=65536), dict(rows=-1), dict(cols=65537), dict(dtype=3),
               dict(out_dtype=2), dict(steps=0), dict(steps=65), dict(a=17.0), dict(b=nan),
               dict(c=inf), dict(eps=-1e-9), dict(eps=nan), dict(eps=inf)):
        assert ortho(**kw) == INVALID, kw
    for kw in (dict(batch=0), dict(rows=0), dict(cols=0)):
        assert ortho(**kw) == OK, kw
    assert ortho() == INVALID                                  # null pointers
    size = lib.beam_moe_orthogonalize_workspace_size
    assert size(1, 64, 512, 3) == 0 and size(-1, 64, 512, 0) == 0
    assert size(8, 2560, 5120, 2) > size(8, 2560, 5120, 0) > 0


def test_binding_refuses_host_tensors():
    """The binding's own checks come before the library is asked."""
    x, w = torch.zeros(4, 8).bfloat16(), torch.zeros(2, 8, 8).bfloat16()
    off = torch.tensor([0, 1, 4], dtype=torch.int32)
    with pytest.raises(TypeError):
        api.grouped_matmul(x, w, off)
    with pytest.raises(TypeError):
        api.grouped_matmul_dw(x, x, off)
    with pytest.raises(TypeError):
        api.swiglu(x, x)
    with pytest.raises(TypeError):
        api.orthogonalize(x)
    with pytest.raises(TypeError):
        api.swiglu(None, x)
    with pytest.raises(ValueError):
        api.grouped_matmul_workspace_size(4, 2000, 8, 8)
    with pytest.raises(TypeError):
        api.grouped_matmul_workspace_size(4, 2, 8, 8, dtype=torch.float32)
