"""Host-side checks of the 8-bit linear layer and of the gradient norm and clipping: bad arguments are refused before
anything is launched (no GPU needed), and the size queries are host-only."""
import ctypes

import pytest

from qlora_quantized_linear_b200 import lbq


def _w(**kw):
    w = lbq.lbq_i8weight(n=256, k=512, codes=0x1000, scale=0x2000)
    for key, v in kw.items():
        setattr(w, key, v)
    return w


WS = 1 << 20

BAD_WEIGHTS = [
    (dict(n=0), lbq.LBQ_EINVAL), (dict(k=0), lbq.LBQ_EINVAL), (dict(k=520), lbq.LBQ_EINVAL), (dict(k=8), lbq.LBQ_EINVAL),
    (dict(k=131088), lbq.LBQ_EINVAL), (dict(codes=None), lbq.LBQ_EINVAL), (dict(scale=None), lbq.LBQ_EINVAL),
    (dict(codes=0x1008), lbq.LBQ_EALIGN), (dict(scale=0x2004), lbq.LBQ_EALIGN),
]


@pytest.mark.parametrize("call", [lbq.lbq_linear_i8_fwd, lbq.lbq_linear_i8_bwd])
@pytest.mark.parametrize("change,expect", BAD_WEIGHTS)
def test_bad_weights(call, change, expect):
    w = _w(**change)
    assert call(0x4000, 4, ctypes.byref(w), None, None, 0, 0.0, 0x5000, None, 0x6000, WS, None) == expect


@pytest.mark.parametrize("call", [lbq.lbq_linear_i8_fwd, lbq.lbq_linear_i8_bwd])
def test_bad_arguments(call):
    w = _w()
    ref = ctypes.byref(w)

    def go(x=0x4000, m=4, q=ref, A=None, B=None, rank=0, y=0x5000, saved=None, ws=0x6000, nws=WS):
        return call(x, m, q, A, B, rank, 1.0, y, saved, ws, nws, None)

    assert go(q=None) == lbq.LBQ_EINVAL
    assert go(x=None) == lbq.LBQ_EINVAL
    assert go(y=None) == lbq.LBQ_EINVAL
    assert go(m=0) == lbq.LBQ_EINVAL
    assert go(m=-1) == lbq.LBQ_EINVAL
    assert go(x=0x4002) == lbq.LBQ_EALIGN
    assert go(y=0x5004) == lbq.LBQ_EALIGN
    assert go(rank=8) == lbq.LBQ_EINVAL                                   # rank > 0 needs A, B and the saved product
    assert go(rank=8, A=0x7000, B=0x8000) == lbq.LBQ_EINVAL
    assert go(rank=65, A=0x7000, B=0x8000, saved=0x9000) == lbq.LBQ_EINVAL
    assert go(rank=-1) == lbq.LBQ_EINVAL
    assert go(rank=8, A=0x7008, B=0x8000, saved=0x9000) == lbq.LBQ_EALIGN
    assert go(ws=None) == lbq.LBQ_EWORKSPACE
    size = lbq.lbq_linear_i8_fwd_workspace_size if call is lbq.lbq_linear_i8_fwd else lbq.lbq_linear_i8_bwd_workspace_size
    assert go(nws=size(4, ref, 0) - 1) == lbq.LBQ_EWORKSPACE
    assert go(ws=0x6008) == lbq.LBQ_EALIGN


@pytest.mark.parametrize("call", [lbq.lbq_linear_i8_fwd, lbq.lbq_linear_i8_bwd])
def test_sixteen_bytes_of_alignment_are_enough(call):
    """Pointers 16 bytes past a 32-byte boundary pass every check up to the workspace, which comes last."""
    w = _w(codes=0x1010, scale=0x2010)
    assert call(0x4010, 4, ctypes.byref(w), 0x7010, 0x8010, 8, 1.0, 0x5010, 0x9010, None, 0, None) == lbq.LBQ_EWORKSPACE
    assert call(0x4010, 4, ctypes.byref(w), 0x7010, 0x8010, 8, 1.0, 0x5010, 0x9010, 0x6008, WS, None) == lbq.LBQ_EALIGN


def test_backward_sizes():
    for n in (100, 131080):                                               # not a multiple of 8; sums past int32
        w = _w(n=n)
        assert lbq.lbq_linear_i8_bwd(0x4000, 4, ctypes.byref(w), None, None, 0, 0.0, 0x5000, None, 0x6000, 1 << 30,
                                     None) == lbq.LBQ_EINVAL


def test_quantize_refuses():
    def go(x=0x4000, dtype=lbq.LBQ_BF16, rows=4, k=64, codes=0x5000, scale=0x6000):
        return lbq.lbq_quantize_i8(x, dtype, rows, k, codes, scale, None)

    for bad in (dict(x=None), dict(codes=None), dict(scale=None), dict(rows=0), dict(k=0), dict(k=24), dict(k=131088)):
        assert go(**bad) == lbq.LBQ_EINVAL
    for bad in (dict(x=0x4008), dict(codes=0x5004), dict(scale=0x6004)):
        assert go(**bad) == lbq.LBQ_EALIGN
    assert go(dtype=3) == lbq.LBQ_EUNSUPPORTED
    assert go(dtype=-1) == lbq.LBQ_EUNSUPPORTED


def test_workspace_sizes():
    w = _w(n=1001, k=2064)
    ref = ctypes.byref(w)
    fwd, bwd = lbq.lbq_linear_i8_fwd_workspace_size, lbq.lbq_linear_i8_bwd_workspace_size
    # codes and a scale per token; the backward's rows are padded to 16 bytes
    assert fwd(77, ref, 5) >= 77 * 2064 + 4 * 77
    assert bwd(77, ref, 5) >= 77 * 1008 + 4 * 77
    assert fwd(0, ref, 0) == 0 and bwd(-3, ref, 0) == 0 and fwd(4, ref, 65) == 0 and fwd(4, None, 0) == 0
    big = _w(n=131072, k=131072)
    assert fwd(1 << 20, ctypes.byref(big), 0) > 1 << 37                   # past 32 bits
    assert lbq.lbq_grad_norm_workspace_size(0) == 0
    assert 0 < lbq.lbq_grad_norm_workspace_size(1) <= lbq.lbq_grad_norm_workspace_size(5000)


def _grads(*rows):
    arr = (lbq.lbq_grad * len(rows))()
    for i, (g, out, numel, dtype) in enumerate(rows):
        arr[i] = lbq.lbq_grad(g=g, out=out, numel=numel, dtype=dtype, reserved=0)
    return arr


def _clip(arr, max_norm=1.0, norm=0x9000, ws=0xA000, nws=WS, count=None):
    return lbq.lbq_clip_grad_norm(arr, len(arr) if count is None else count, max_norm, norm, ws, nws, None)


def test_gradient_lists_refuse():
    ok = _grads((0x10000, 0x10000, 100, lbq.LBQ_F32))
    assert _clip(ok, count=0) == lbq.LBQ_EINVAL
    assert lbq.lbq_clip_grad_norm(None, 1, 1.0, 0x9000, 0xA000, WS, None) == lbq.LBQ_EINVAL
    assert _clip(ok, norm=None) == lbq.LBQ_EINVAL
    assert _clip(ok, norm=0x9004) == lbq.LBQ_EALIGN
    for bad in (-0.5, float("nan"), float("inf")):
        assert _clip(ok, max_norm=bad) == lbq.LBQ_EINVAL
    assert _clip(ok, ws=None) == lbq.LBQ_EWORKSPACE
    assert _clip(ok, nws=lbq.lbq_grad_norm_workspace_size(1) - 1) == lbq.LBQ_EWORKSPACE
    assert _clip(ok, ws=0xA008) == lbq.LBQ_EALIGN
    assert _clip(_grads((None, 0x10000, 100, lbq.LBQ_F32))) == lbq.LBQ_EINVAL
    assert _clip(_grads((0x10000, None, 100, lbq.LBQ_F32))) == lbq.LBQ_EINVAL
    assert _clip(_grads((0x10000, 0x10000, -1, lbq.LBQ_F32))) == lbq.LBQ_EINVAL
    assert _clip(_grads((0x10000, 0x10000, 100, 3))) == lbq.LBQ_EUNSUPPORTED
    assert _clip(_grads((0x10002, 0x10002, 100, lbq.LBQ_F32))) == lbq.LBQ_EALIGN
    assert _clip(_grads((0x10001, 0x10001, 100, lbq.LBQ_BF16))) == lbq.LBQ_EALIGN
    assert _clip(_grads((0x10000, 0x20002, 100, lbq.LBQ_F32))) == lbq.LBQ_EALIGN
    assert lbq.lbq_grad_norm(_grads((None, None, 5, lbq.LBQ_F32)), 1, 0x9000, 0xA000, WS, None) == lbq.LBQ_EINVAL


def test_overlapping_gradients_refuse():
    F, H = lbq.LBQ_F32, lbq.LBQ_BF16
    for rows in (
        [(0x10000, 0x10000, 100, F), (0x10000, 0x10000, 100, F)],                       # the same tensor twice
        [(0x10000, 0x10000, 100, F), (0x10000 + 396, 0x10000 + 396, 10, F)],            # a shared last element
        [(0x20000, 0x20000, 8, H), (0x10000, 0x10000, 0x8001, H), (0x30000, 0x30000, 8, H)],  # unsorted, one byte pair over
        [(0x10000, 0x20000, 100, F), (0x20000, 0x30000, 100, F)],                       # an output over a later input
        [(0x20000, 0x30000, 100, F), (0x10000, 0x20000 + 396, 100, F)],                 # its first element, unsorted
        [(0x10000, 0x10004, 100, F)],                                                   # shifted onto itself
        [(0x10000, 0x0FFFC, 100, F)],
    ):
        assert _clip(_grads(*rows)) == lbq.LBQ_EINVAL, rows
