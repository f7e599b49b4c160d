"""Host side of the gradient-making operators: sizes, and the refusals that
come before any device work (the library is called with stand-in addresses that
no refused call touches)."""
import ctypes

import pytest
import torch

from error_compensated_bit_02_amd import ActCheckpoint, OneBitError, act_layout, binding

P = 1 << 20            # a stand-in device address, aligned to 16 bytes
INVALID, ALIGN = 1, 2


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


@pytest.mark.parametrize("rows,cols,want", [
    (0, 1, (64, 0, 0)), (1, 1, (64, 64, 64)), (32, 64, (64, 2048, 64)), (33, 65, (128, 33 * 128, 256)),
    (16384, 8192, (8192, 16384 * 8192, 512 * 8192))])
def test_layout(lib, rows, cols, want):
    assert act_layout(rows, cols) == want


def test_layout_refusals(lib):
    for rows, cols in [(-1, 4), (4, 0), (4, -1), (4, (1 << 30) + 1), ((1 << 31) + 1, 4), (1 << 31, 1 << 30)]:
        with pytest.raises(OneBitError) as e:
            act_layout(rows, cols)
        assert e.value.status == INVALID
    assert lib.ob_act_layout(1, 1, None, None, None) == INVALID


def _save(lib, **k):
    a = dict(fmt=0, fn=1, rows=4, cols=8, dtype=0, x=P, ldx=8, y=P, ldy=8, codes=P, scales=P)
    a.update(k)
    return lib.ob_act_save(a["fmt"], a["fn"], a["rows"], a["cols"], a["dtype"], a["x"], a["ldx"], a["y"], a["ldy"],
                           a["codes"], a["scales"], None)


def test_save_refusals(lib):
    for bad in [dict(fmt=2), dict(fmt=-1), dict(fn=4), dict(fn=-1), dict(rows=-1), dict(cols=0), dict(dtype=2),
                dict(ldx=7), dict(ldy=7), dict(x=None), dict(y=None), dict(fn=0), dict(codes=None),
                dict(scales=None), dict(ldx=1 << 60)]:
        assert _save(lib, **bad) == INVALID, bad
    for bad in [dict(x=P + 2), dict(y=P + 1), dict(dtype=1, x=P + 1), dict(codes=P + 8), dict(scales=P + 4)]:
        assert _save(lib, **bad) == ALIGN, bad
    assert _save(lib, rows=0, x=None, y=None, codes=None, scales=None) == 0     # nothing to do


def test_load_and_backward_refusals(lib):
    def load(fmt=0, rows=4, cols=8, codes=P, scales=P, dtype=0, out=P, ldo=8):
        return lib.ob_act_load(fmt, rows, cols, codes, scales, dtype, out, ldo, None)

    def back(fmt=0, fn=1, rows=4, cols=8, codes=P, scales=P, dtype=0, dy=P, lddy=8, dx=P, lddx=8):
        return lib.ob_act_backward(fmt, fn, rows, cols, codes, scales, dtype, dy, lddy, dx, lddx, None)

    for bad in [dict(fmt=3), dict(rows=-1), dict(cols=0), dict(codes=None), dict(scales=None), dict(dtype=5)]:
        assert load(**bad) == INVALID and back(**bad) == INVALID, bad
    assert load(out=None) == INVALID and load(ldo=7) == INVALID
    assert back(fn=0) == INVALID and back(dy=None) == INVALID and back(dx=None) == INVALID
    assert back(lddy=7) == INVALID and back(lddx=7) == INVALID
    assert load(codes=P + 8) == ALIGN and back(scales=P + 8) == ALIGN and back(dtype=1, dx=P + 1) == ALIGN
    assert load(rows=0, codes=None, scales=None, out=None) == 0
    assert back(rows=0, codes=None, scales=None, dy=None, dx=None) == 0


def test_work_sizes(lib):
    n = ctypes.c_int64()
    for tokens, dim in [(0, 8), (1, 1), (4096, 1024), (4097, 8), (1 << 20, 64)]:
        assert lib.ob_embedding_grad_work(tokens, dim, ctypes.byref(n)) == 0 and n.value >= 8 * tokens
    for tokens, dim in [(-1, 8), (4, 0), (1 << 24, 8), (1 << 23, 1 << 14)]:
        assert lib.ob_embedding_grad_work(tokens, dim, ctypes.byref(n)) == INVALID
    for rows, out, inp in [(0, 1, 1), (1, 1, 1), (4096, 1024, 1024), (1 << 24, 64, 64)]:
        assert lib.ob_linear_grad_work(rows, out, inp, 1, 1, ctypes.byref(n)) == 0 and n.value >= 0
    for rows, out, inp, dt in [(-1, 4, 4, 0), (4, 0, 4, 0), (4, 4, 0, 0), (4, 4, 4, 2), ((1 << 24) + 1, 4, 4, 0),
                               (4, 4, (1 << 24) + 1, 0), (4, 1 << 30, 1 << 24, 0)]:
        assert lib.ob_linear_grad_work(rows, out, inp, dt, 0, ctypes.byref(n)) == INVALID
    assert lib.ob_embedding_grad_work(1, 1, None) == INVALID
    assert lib.ob_linear_grad_work(1, 1, 1, 0, 0, None) == INVALID


def test_calls_without_a_context_are_refused(lib):
    assert lib.ob_embedding_lookup(None, 0, 8, 1, P, 0, P, 1.0, 0, P, 8, None) == INVALID
    assert lib.ob_embedding_grad(None, 0, 0, 8, 1, P, 0, 1.0, 0, P, 8, 0, P, P, 1 << 20, None) == INVALID
    assert lib.ob_linear_grad(None, 0, 0, -1, 1, 8, 8, 0, P, P, 0, P, 8, 0, P, P, 1 << 20, None) == INVALID


def test_binding_refuses_host_tensors_and_bad_names():
    with pytest.raises(OneBitError, match="device tensor"):
        ActCheckpoint(4, 8, codes=torch.zeros(4, 64, dtype=torch.uint8), scales=torch.zeros(1, 64, dtype=torch.uint8))
    with pytest.raises(OneBitError, match="format"):
        ActCheckpoint(4, 8, "e5m2")
    with pytest.raises(OneBitError, match="together"):
        ActCheckpoint(4, 8, codes=torch.zeros(4, 64, dtype=torch.uint8))
