"""GPU checks of sp24_quantize_rows against the IEEE fp32 operations of its definition (numpy),
bit for bit, and against the 64-bit bound |q scale - x| <= scale (1/2 + 2^-14): rint is off by
at most 1/2, and 1/amax, its product with 127, the product with x and amax/127 each by 2^-24
relative (1/amax by 2^-23 where it is subnormal) of at most 127."""
import numpy as np
import pytest
import torch

import oracle
import structured_sparse_transformer_b200 as sp
import synthetic_inputs as si

pytestmark = pytest.mark.gpu


def _reference(x, keep=None):
    """x: fp16/bf16 CPU tensor -> (q, scale) by the definition."""
    v = x.float().numpy().copy()
    if keep is not None:
        v[~keep] = 0.0
    with np.errstate(all="ignore"):
        amax = np.abs(v).max(axis=1) if v.shape[1] else np.zeros(v.shape[0], np.float32)
        bad = ~np.isfinite(amax)
        small = ~bad & (amax < np.float32(2.0**-100))
        inv = np.where(bad | small, np.float32(0), (np.float32(1) / amax) * np.float32(127)).astype(np.float32)
        scale = np.where(bad, np.float32("nan"), np.where(small, np.float32(0), amax / np.float32(127)))
        prod = (v * inv[:, None]).astype(np.float32)
        q = np.where(inv[:, None] == 0, 0, np.rint(np.where(np.isfinite(prod), prod, 0)))
    return q.astype(np.int8), scale.astype(np.float32)


def _run(xd, idx=None):
    R, C = xd.shape
    q = torch.full((R + 1, C), 77, dtype=torch.int8, device="cuda")
    s = torch.full((R + 1,), -5.0, device="cuda")
    sp.sp24_quantize_rows(xd, q, s, idx)
    torch.cuda.synchronize()
    assert (q[R:] == 77).all() and (s[R:] == -5.0).all()      # nothing behind the last row
    return q[:R].cpu().numpy(), s[:R].cpu().numpy()


def _check(xd, idx=None, keep=None):
    q, s = _run(xd, idx)
    qr, sr = _reference(xd.cpu(), keep)
    assert np.array_equal(s.view(np.uint32) & 0x7FFFFFFF, sr.view(np.uint32) & 0x7FFFFFFF) or \
        (np.array_equal(np.isnan(s), np.isnan(sr)) and np.array_equal(s[~np.isnan(s)], sr[~np.isnan(sr)]))
    assert np.array_equal(q, qr)
    return q, s


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 16), (3, 7), (5, 31), (1, 1600), (2, 2048), (33, 1000), (7, 5120), (4, 6400),
                                 (9, 16392), (2, 40001), (300, 64)])
def test_rows_of_any_size(R, C, dtype):
    x = si.normal((R, C), 1.0, R * 7 + C, dtype)
    q, s = _check(x.cuda())
    err = np.abs(q.astype(np.float64) * s[:, None] - x.double().numpy())
    assert (err <= s[:, None].astype(np.float64) * (0.5 + 2.0**-14)).all()


@pytest.mark.parametrize("pitch", [0, 1, 8, 13])
@pytest.mark.parametrize("C", [24, 2048, 515])
def test_row_pitch(pitch, C):
    x = si.normal((17, C + pitch), 3.0, C, "bf16").cuda()
    _check(x[:, :C])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("R,C", [(4, 4), (8, 12), (64, 128), (100, 404), (256, 1600), (8, 8200)])
def test_masked_weight(R, C, dtype):
    w = si.normal((R, C), 0.02, R + C, dtype)
    idx = oracle.mask_search(si.bits16(w), dtype)
    keep = oracle.dense_mask(idx).astype(bool)
    # what a pruned place holds does not matter: NaN, infinities and the largest values
    for k, junk in enumerate((float("nan"), float("inf"), -float("inf"), torch.finfo(w.dtype).max)):
        at = torch.from_numpy(~keep) & (torch.arange(R * C).reshape(R, C) % 4 == k)
        w[at] = junk
    _check(w.cuda(), torch.from_numpy(idx).cuda(), keep)


def test_rows_with_nothing_or_too_much():
    for dt in (torch.float16, torch.bfloat16):
        x = torch.randn(8, 160, generator=torch.Generator().manual_seed(3)).to(dt)
        x[0] = 0
        x[1] = -0.0
        x[2, 5] = float("nan")
        x[3, 159] = float("inf")
        x[4, 0] = -float("inf")
        x[5] = torch.finfo(dt).smallest_normal * 2.0**-3       # fp16: a normal row; bf16: below 2^-100
        x[6] = torch.finfo(dt).max
        x[7] = 0
        x[7, 100] = torch.finfo(dt).tiny
        _check(x.cuda())


def test_ties_go_to_even():
    x = torch.zeros(1, 64, dtype=torch.float16)
    x[0, 0] = 127.0
    x[0, 1:33] = torch.arange(32) + 0.5
    q, s = _check(x.cuda())
    assert s[0] == 1.0 and q[0, 1] == 0 and q[0, 2] == 2 and q[0, 3] == 2 and q[0, 4] == 4


def test_zero_sizes_streams_and_repeats():
    q, s = torch.zeros(0, 8, dtype=torch.int8, device="cuda"), torch.zeros(0, device="cuda")
    sp.sp24_quantize_rows(torch.zeros(0, 8, dtype=torch.float16, device="cuda"), q, s)
    s3 = torch.ones(3, device="cuda")
    sp.sp24_quantize_rows(torch.zeros(3, 0, dtype=torch.float16, device="cuda"), torch.zeros(3, 0, dtype=torch.int8,
                                                                                          device="cuda"), s3)
    assert (s3 == 0).all()
    x = si.normal((64, 1600), 1.0, 5, "f16").cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for _ in range(2):
        q, s = torch.empty(64, 1600, dtype=torch.int8, device="cuda"), torch.empty(64, device="cuda")
        sp.sp24_quantize_rows(x, q, s, stream=side)
        outs.append((q, s))
    side.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert np.array_equal(outs[0][0].cpu().numpy(), _reference(x.cpu())[0])


@pytest.mark.parametrize("rows,cols", [(70001, 32768), (524289, 4104)])
def test_matrices_past_32_bit_offsets(rows, cols):
    """More than 2^31 entries: the last rows are as in a small call."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    q, s = torch.empty(rows, cols, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    sp.sp24_quantize_rows(x, q, s)
    for lo in (0, rows // 2, rows - 4):
        qr, sr = _reference(x[lo:lo + 4].cpu())
        assert np.array_equal(q[lo:lo + 4].cpu().numpy(), qr) and np.array_equal(s[lo:lo + 4].cpu().numpy(), sr)
