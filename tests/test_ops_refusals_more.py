"""More argument checks of the optimiser-step and 8-bit entry points (no device needed)."""
import ctypes

import pytest
import torch

import structured_sparse_transformer_b200 as sp

E = {v: k for k, v in sp.STATUS.items()}
F = ctypes.c_float
A = [ctypes.c_void_p(0x10000000 * (k + 1)) for k in range(6)]      # far from one another


def _raw(name, *args):
    return getattr(sp.lib(), name)(*args)


def _off(p, by):
    return ctypes.c_void_p(p.value + by)


def _i8(x=A[0], sx=A[1], T=32, K=64, w=A[2], sw=A[3], N=64, y=A[4]):
    return _raw("sp24_gemm_i8", x, sx, T, K, w, sw, N, 0, y, 0, None)


def _quant(x=A[0], rows=32, cols=64, ldx=64, idx=None, q=A[1], scale=A[2]):
    return _raw("sp24_quantize_rows", x, 0, rows, cols, ldx, idx, q, scale, None)


@pytest.mark.parametrize("by", [1, 2, 3])
def test_scales_at_odd_addresses_are_refused(by):
    """A 4-byte access at such an address would fault."""
    assert _i8(sx=_off(A[1], by)) == _i8(sw=_off(A[3], by)) == E["SP24_ERR_MISALIGNED"]
    assert _quant(scale=_off(A[2], by)) == _quant(cols=0, ldx=0, scale=_off(A[2], by)) == E["SP24_ERR_MISALIGNED"]


def test_scales_at_word_addresses_are_taken():
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert _i8(sx=_off(A[1], 4), sw=_off(A[3], 8)) == _quant(scale=_off(A[2], 12)) == E["SP24_ERR_NO_DEVICE"]


def test_matrices_of_other_rows_are_refused():
    """Right in size, but of other rows: a transposed result would hold other entries, a transposed mask prune others.
    Flat buffers, and more rows than needed, are taken (and stop at the device check)."""
    T, K, N = 32, 16, 64
    xq, wq = torch.zeros(T, K, dtype=torch.int8), torch.zeros(N, K, dtype=torch.int8)
    for shape, why in (((N, T), "rows of 64"), ((1, N, T), "rows of 64"), ((T * N // 16, 16), "rows of 64"),
                       ((T * N,), "CUDA"), ((T + 2, N), "CUDA"), ((2, T // 2, N), "CUDA"), ((T, N), "CUDA")):
        with pytest.raises(ValueError, match=why):
            sp.sp24_gemm_i8(xq, torch.zeros(T), wq, torch.zeros(N), torch.zeros(shape, dtype=torch.float16))
    R, C = 32, 64
    x, s = torch.zeros(R, C, dtype=torch.float16), torch.zeros(R)
    for shape, why in (((C, R), "q: expected rows of 64"), ((R * C,), "CUDA"), ((R + 1, C), "CUDA")):
        with pytest.raises(ValueError, match=why):
            sp.sp24_quantize_rows(x, torch.zeros(shape, dtype=torch.int8), s)
    q = torch.zeros(R, C, dtype=torch.int8)
    for shape, why in (((C // 4, R // 4), "idx: expected rows of 16"), ((R * C // 16,), "CUDA"), ((R // 4, C // 4), "CUDA")):
        with pytest.raises(ValueError, match=why):
            sp.sp24_quantize_rows(x, q, s, torch.zeros(shape, dtype=torch.uint8))


def test_the_largest_sizes():
    """The limits that the header names, just inside and just past them."""
    def size(count, rows, cols):
        return _raw("sp24_orthogonalize_size", count, rows, cols, ctypes.byref(ctypes.c_size_t(0)))

    for inside in ((1, 1 << 24, 4), (1, 4, 1 << 24), (1, 65536, 1 << 24), (65535, 4, 4), (65535, 8192, 4096), (1, 65536, 65536)):
        assert size(*inside) == E["SP24_OK"], inside
    for past in ((1, (1 << 24) + 1, 4), (1, 4, (1 << 24) + 1), (65536, 4, 4), (1, 65537, 65537), (65535, 65536, 65536)):
        assert size(*past) == E["SP24_ERR_UNSUPPORTED_SHAPE"], past
