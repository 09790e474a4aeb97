"""Argument checks of the optimiser-step and 8-bit entry points (no device needed): the C
calls' status codes, and the binding's checks of layout, dtype, size and device."""
import ctypes

import numpy as np
import pytest
import torch

import structured_sparse_transformer_b200 as sp

E = {v: k for k, v in sp.STATUS.items()}
FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)
HALF, BYTE = ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10001)
F = ctypes.c_float


def _raw(name, *args):
    return getattr(sp.lib(), name)(*args)


@pytest.mark.parametrize("count,rows,cols", [(1, 1, 1), (1, 512, 256), (3, 451, 317), (8, 4096, 1024), (1, 1600, 6400)])
def test_workspace_size_covers_its_parts(count, rows, cols):
    m, n = sorted((rows, cols))
    pad = lambda v: -(-v // 8) * 8
    need = 2 * (2 * count * m * pad(n)) + 2 * (2 * count * m * pad(m))
    got = sp.sp24_orthogonalize_size(rows, cols, count)
    assert need <= got <= need + count * (1 << 16) + 2 * 80 * (1 << 17) + (1 << 16)   # + split tiles' partial sums
    assert sp.sp24_orthogonalize_size(cols, rows, count) == got


def test_sizes_that_are_not_taken():
    assert sp.sp24_orthogonalize_size(0, 64) == sp.sp24_orthogonalize_size(64, 64, 0) == 0
    for args in ((-1, 64, 64), (1, -1, 64), (1, 64, -1)):
        out = ctypes.c_size_t(0)
        assert _raw("sp24_orthogonalize_size", *args, ctypes.byref(out)) == E["SP24_ERR_INVALID_ARG"]
    out = ctypes.c_size_t(0)
    assert _raw("sp24_orthogonalize_size", 1, 70000, 70000, ctypes.byref(out)) == E["SP24_ERR_UNSUPPORTED_SHAPE"]
    assert _raw("sp24_orthogonalize_size", 70000, 4, 4, ctypes.byref(out)) == E["SP24_ERR_UNSUPPORTED_SHAPE"]
    assert _raw("sp24_orthogonalize_size", 1, 4, 4, None) == E["SP24_ERR_INVALID_ARG"]


def _orth(G=FAKE, count=1, rows=64, cols=32, ld=32, stride=2048, steps=5, eps=1e-7, out=FAKE, dt=0, ws=FAKE,
          ws_bytes=1 << 30):
    return _raw("sp24_orthogonalize", G, count, rows, cols, ld, stride, steps, F(eps), out, dt, ws, ws_bytes, None)


def _muon(g=FAKE, m=FAKE, w=FAKE, w16=FAKE, dt=0, count=1, rows=64, cols=32, steps=5, eps=1e-7, ws=FAKE,
          ws_bytes=1 << 30):
    return _raw("sp24_muon_step", g, m, w, w16, dt, count, rows, cols, F(0.95), 1, F(0.02), F(0.1), F(1.0), steps,
                F(eps), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(G=None), "SP24_ERR_INVALID_ARG"), (dict(out=None), "SP24_ERR_INVALID_ARG"),
    (dict(ws=None), "SP24_ERR_INVALID_ARG"), (dict(rows=-1), "SP24_ERR_INVALID_ARG"),
    (dict(ld=31), "SP24_ERR_INVALID_ARG"), (dict(stride=-1), "SP24_ERR_INVALID_ARG"),
    (dict(steps=0), "SP24_ERR_INVALID_ARG"), (dict(steps=17), "SP24_ERR_INVALID_ARG"),
    (dict(eps=-1e-3), "SP24_ERR_INVALID_ARG"), (dict(eps=float("nan")), "SP24_ERR_INVALID_ARG"),
    (dict(dt=5), "SP24_ERR_UNSUPPORTED_DTYPE"), (dict(G=HALF), "SP24_ERR_MISALIGNED"),
    (dict(out=BYTE), "SP24_ERR_MISALIGNED"), (dict(ws=ODD), "SP24_ERR_MISALIGNED"),
    (dict(ws_bytes=1000), "SP24_ERR_SCRATCH_TOO_SMALL"), (dict(count=70000), "SP24_ERR_UNSUPPORTED_SHAPE")])
def test_orthogonalize_refuses(kw, status):
    assert _orth(**kw) == E[status]


@pytest.mark.parametrize("kw,status", [
    (dict(g=None), "SP24_ERR_INVALID_ARG"), (dict(m=None), "SP24_ERR_INVALID_ARG"),
    (dict(w=None), "SP24_ERR_INVALID_ARG"), (dict(cols=-4), "SP24_ERR_INVALID_ARG"),
    (dict(steps=0), "SP24_ERR_INVALID_ARG"), (dict(dt=2), "SP24_ERR_UNSUPPORTED_DTYPE"),
    (dict(g=HALF), "SP24_ERR_MISALIGNED"), (dict(m=HALF), "SP24_ERR_MISALIGNED"), (dict(w=HALF), "SP24_ERR_MISALIGNED"),
    (dict(w16=BYTE), "SP24_ERR_MISALIGNED"), (dict(ws_bytes=16), "SP24_ERR_SCRATCH_TOO_SMALL")])
def test_muon_step_refuses(kw, status):
    assert _muon(**kw) == E[status]


@pytest.mark.parametrize("args,status", [
    ((None, 0, 4, 8, 8, None, FAKE, FAKE, None), "SP24_ERR_INVALID_ARG"),
    ((FAKE, 0, 4, 8, 8, None, None, FAKE, None), "SP24_ERR_INVALID_ARG"),
    ((FAKE, 0, 4, 8, 8, None, FAKE, None, None), "SP24_ERR_INVALID_ARG"),
    ((FAKE, 0, 4, 8, 7, None, FAKE, FAKE, None), "SP24_ERR_INVALID_ARG"),
    ((FAKE, 0, -4, 8, 8, None, FAKE, FAKE, None), "SP24_ERR_INVALID_ARG"),
    ((FAKE, 3, 4, 8, 8, None, FAKE, FAKE, None), "SP24_ERR_UNSUPPORTED_DTYPE"),
    ((FAKE, 0, 6, 8, 8, FAKE, FAKE, FAKE, None), "SP24_ERR_UNSUPPORTED_SHAPE"),
    ((FAKE, 0, 4, 6, 8, FAKE, FAKE, FAKE, None), "SP24_ERR_UNSUPPORTED_SHAPE"),
    ((ODD, 0, 4, 8, 8, None, FAKE, FAKE, None), "SP24_ERR_MISALIGNED"),
    ((FAKE, 0, 4, 8, 8, None, ODD, FAKE, None), "SP24_ERR_MISALIGNED")])
def test_quantize_rows_refuses(args, status):
    assert _raw("sp24_quantize_rows", *args) == E[status]


def _i8(x=FAKE, sx=FAKE, T=32, K=64, w=FAKE, sw=FAKE, N=64, dt=0, y=FAKE, epi=0):
    return _raw("sp24_gemm_i8", x, sx, T, K, w, sw, N, dt, y, epi, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), "SP24_ERR_INVALID_ARG"), (dict(sx=None), "SP24_ERR_INVALID_ARG"),
    (dict(w=None), "SP24_ERR_INVALID_ARG"), (dict(sw=None), "SP24_ERR_INVALID_ARG"),
    (dict(y=None), "SP24_ERR_INVALID_ARG"), (dict(T=-1), "SP24_ERR_INVALID_ARG"), (dict(K=0), "SP24_ERR_INVALID_ARG"),
    (dict(N=0), "SP24_ERR_INVALID_ARG"), (dict(K=40), "SP24_ERR_UNSUPPORTED_SHAPE"),
    (dict(N=40), "SP24_ERR_UNSUPPORTED_SHAPE"), (dict(K=131072), "SP24_ERR_UNSUPPORTED_SHAPE"),
    (dict(dt=7), "SP24_ERR_UNSUPPORTED_DTYPE"), (dict(epi=2), "SP24_ERR_INVALID_ARG"),
    (dict(epi=6), "SP24_ERR_INVALID_ARG"), (dict(x=ODD), "SP24_ERR_MISALIGNED"), (dict(w=ODD), "SP24_ERR_MISALIGNED"),
    (dict(y=ODD), "SP24_ERR_MISALIGNED")])
def test_gemm_i8_refuses(kw, status):
    assert _i8(**kw) == E[status]


def test_the_longest_contraction_cannot_overflow():
    K = 131056
    assert K % 16 == 0 and K * 128 * 128 <= 2**31 - 1 < (K + 16) * 128 * 128


def test_binding_checks_come_before_the_device_check():
    """CPU tensors: a call whose arguments are right stops at the device check; every wrong one before it."""
    f32, f16, i8, u8 = torch.float32, torch.float16, torch.int8, torch.uint8
    g = torch.zeros(64, 32, dtype=f32)
    o = torch.zeros(64, 32, dtype=f16)
    ws = torch.zeros(sp.sp24_orthogonalize_size(64, 32), dtype=u8)

    def bad(fn, *a, match, exc=ValueError, **kw):
        with pytest.raises(exc, match=match):
            fn(*a, **kw)

    bad(sp.sp24_orthogonalize, g, o, ws, match="CUDA")
    bad(sp.sp24_orthogonalize, torch.zeros(64, 48)[:, :32], o, ws, match="CUDA")     # a row pitch is fine
    bad(sp.sp24_orthogonalize, g.t(), o, ws, match="unit stride")
    bad(sp.sp24_orthogonalize, g[0], o, ws, match="matrix or a stack")
    bad(sp.sp24_orthogonalize, g.double(), o, ws, match="G:")
    bad(sp.sp24_orthogonalize, g, o.float(), ws, match="dtype", exc=TypeError)
    bad(sp.sp24_orthogonalize, g, o[:63], ws, match="out")
    bad(sp.sp24_orthogonalize, g, o, ws[:-1], match="workspace")
    bad(sp.sp24_orthogonalize, g, o, ws.to(i8), match="workspace")
    m, w = torch.zeros_like(g), torch.zeros_like(g)
    bad(sp.sp24_muon_step, g, m, w, o, ws, lr=0.1, match="CUDA")
    bad(sp.sp24_muon_step, g, m, w, None, ws, lr=0.1, match="CUDA")
    bad(sp.sp24_muon_step, g.t().contiguous(), m, w, o, ws, lr=0.1, match="grad: expected shape")
    bad(sp.sp24_muon_step, g.half(), m, w, o, ws, lr=0.1, match="grad")
    bad(sp.sp24_muon_step, g, m[:3], w, o, ws, lr=0.1, match="momentum")
    bad(sp.sp24_muon_step, g, m, w, o[:3], ws, lr=0.1, match="W16")
    bad(sp.sp24_muon_step, g, m, w, o, ws[:9], lr=0.1, match="workspace")
    x = torch.zeros(8, 16, dtype=f16)
    q, s = torch.zeros(8, 16, dtype=i8), torch.zeros(8)
    idx = torch.zeros(2, 4, dtype=u8)
    bad(sp.sp24_quantize_rows, x, q, s, match="CUDA")
    bad(sp.sp24_quantize_rows, x, q, s, idx, match="CUDA")
    bad(sp.sp24_quantize_rows, x.t(), q, s, match="row-major")
    bad(sp.sp24_quantize_rows, x.float(), q, s, match="dtype", exc=TypeError)
    bad(sp.sp24_quantize_rows, x, q[:7], s, match="q:")
    bad(sp.sp24_quantize_rows, x, q.to(u8), s, match="q:")
    bad(sp.sp24_quantize_rows, x, q, s[:7], match="scale")
    bad(sp.sp24_quantize_rows, x, q, s, idx[:1], match="idx")
    wq, sw, y = torch.zeros(32, 16, dtype=i8), torch.zeros(32), torch.zeros(8, 32, dtype=f16)
    bad(sp.sp24_gemm_i8, q, s, wq, sw, y, match="CUDA")
    bad(sp.sp24_gemm_i8, q, s, wq[:, :8].contiguous(), sw, y, match="columns")
    bad(sp.sp24_gemm_i8, q, s[:3], wq, sw, y, match="sx")
    bad(sp.sp24_gemm_i8, q, s, wq, sw[:3], y, match="sw")
    bad(sp.sp24_gemm_i8, q, s, wq, sw, y[:3], match="Y")
    bad(sp.sp24_gemm_i8, q, s, wq, sw, y.float(), match="dtype", exc=TypeError)
    bad(sp.sp24_gemm_i8, q.to(u8), s, wq, sw, y, match="Xq")


def test_valid_calls_without_a_device_report_no_device():
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert _orth() == _muon() == _i8() == E["SP24_ERR_NO_DEVICE"]
    assert _raw("sp24_quantize_rows", FAKE, 0, 4, 8, 8, None, FAKE, FAKE, None) == E["SP24_ERR_NO_DEVICE"]


def test_tile_numbering_of_the_symmetric_products():
    """Every block on and below the diagonal once, none above: the kernel's numbering restated."""
    for m in (1, 100, 128, 129, 256, 257, 700, 1600, 5000):
        for bn in (128, 256):
            R, rb, cb = 256 // bn, -(-m // 256), -(-m // bn)
            total = R * rb * (rb - 1) // 2 + min(cb, R * rb)
            seen = set()
            for t in range(total):
                i = int((np.sqrt(np.float32(1 + 8 * t / R)) - 1) * 0.5)
                while R * i * (i + 1) // 2 > t:
                    i -= 1
                while R * (i + 1) * (i + 2) // 2 <= t:
                    i += 1
                seen.add((i, t - R * i * (i + 1) // 2))
            want = {(i, j) for i in range(rb) for j in range(cb) if j * bn < (i + 1) * 256}
            assert seen == want and len(seen) == total


@pytest.mark.parametrize("call,kw", [(_orth, dict(eps=float("inf"))), (_muon, dict(eps=float("inf")))])
def test_an_infinite_eps_is_refused(call, kw):
    assert call(**kw) == E["SP24_ERR_INVALID_ARG"]


def test_results_of_other_rows_are_refused():
    """Right in size, but of other rows: a transposed result would hold other entries.  (A flat buffer is taken.)"""
    g, ws = torch.zeros(64, 32), torch.zeros(sp.sp24_orthogonalize_size(64, 32), dtype=torch.uint8)
    for shape, why in (((32, 64), "rows of 32"), ((1, 32, 64), "rows of 32"), ((2048,), "CUDA"), ((1, 64, 32), "CUDA")):
        o = torch.zeros(shape, dtype=torch.float16)
        with pytest.raises(ValueError, match=why):
            sp.sp24_orthogonalize(g, o, ws)
        with pytest.raises(ValueError, match=why):
            sp.sp24_muon_step(g, g.clone(), g.clone(), o, ws, lr=0.1)
