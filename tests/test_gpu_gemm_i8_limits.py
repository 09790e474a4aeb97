"""GPU checks of sp24_gemm_i8 at the ends of the number range, in every form of the product (dot products, split K, pairs)."""
import pytest
import torch

import structured_sparse_transformer_b200 as sp

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _product(xq, sx, wq, sw, dt, epi):
    y = torch.empty(xq.shape[0], wq.shape[0], dtype=dt, device="cuda")
    sp.sp24_gemm_i8(xq.cuda(), sx.cuda(), wq.cuda(), sw.cuda(), y, epi)
    torch.cuda.synchronize()
    assert sp.sp24_device_status() == 0
    return y.cpu()


@pytest.mark.parametrize("T", [1, 2, 5, 40, 100, 700])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("epi", [None, "gelu"])
def test_products_past_the_range_are_infinite(T, dtype, epi):
    """Scales of 1e20 each: the product of 1e46 and more is infinite in fp32, and gelu takes it to infinity or to 0; a
    token with a NaN scale is NaN, one with a zero scale 0, and the tokens beside them are as without."""
    K, N = 1600, 272
    g = torch.Generator().manual_seed(T)
    xq = torch.randint(1, 128, (T, K), generator=g).to(torch.int8)
    wq = torch.randint(1, 128, (N, K), generator=g).to(torch.int8)
    wq[1::2] = -wq[1::2]
    sx, sw = torch.full((T,), 1e20), torch.full((N,), 1e20)
    special = T > 2
    if special:
        sx[0], sx[2] = float("nan"), 0.0
    y = _product(xq, sx, wq, sw, DT[dtype], epi).float()
    rows = [t for t in range(T) if not (special and t in (0, 2))]
    assert (y[rows][:, ::2] == float("inf")).all()
    assert (y[rows][:, 1::2] == (0.0 if epi else -float("inf"))).all()
    if special:
        assert torch.isnan(y[0]).all()
        assert (y[2] == 0).all()


@pytest.mark.parametrize("T", [1, 5, 40, 700])
def test_the_largest_finite_products(T):
    """Just inside fp32's range and past fp16's: infinite in fp16 by rounding, the rounded value in bf16."""
    K, N = 64, 48
    xq, wq = torch.ones(T, K, dtype=torch.int8), torch.ones(N, K, dtype=torch.int8)
    wq[1::2] = -1
    sx, sw = torch.full((T,), 2.0**60), torch.full((N,), 2.0**61)       # 64 2^121 = 2^127
    for epi in (None, "gelu"):
        y = _product(xq, sx, wq, sw, torch.bfloat16, epi).double()
        assert (y[:, ::2] == 2.0**127).all() and (y[:, 1::2] == (0.0 if epi else -2.0**127)).all()
        y = _product(xq, sx, wq, sw, torch.float16, epi).double()
        assert (y[:, ::2] == float("inf")).all() and (y[:, 1::2] == (0.0 if epi else -float("inf"))).all()


@pytest.mark.parametrize("T", [1, 5, 40, 700])
def test_the_far_tail_of_gelu(T):
    """x from -5.7 to -12, where gelu(x) is 1e-8 and less: |x| R(|x| / sqrt 2) with R(z) = erfc(z) exp(z^2) lies between
    its values at 4 sqrt 2 (0.9713 of its limit sqrt(2/pi)) and at infinity, so the
    clamped factor is at most 1 - 0.9713 = 2.9% off; exp's argument of up to 72 in fp32 adds 72 (2^-23) 2, its
    argument in base 2 up to 104; and bf16's rounding 2^-8."""
    K, N = 16, 128
    xq, wq = torch.zeros(T, K, dtype=torch.int8), torch.zeros(N, K, dtype=torch.int8)
    xq[:, 0] = 1
    wq[:, 0] = -torch.arange(N).to(torch.int8)
    sx, sw = torch.ones(T), torch.full((N,), 12.0 / 127.0)
    y = _product(xq, sx, wq, sw, torch.bfloat16, "gelu").double()
    x = -torch.arange(N).double() * sw.double()
    ref = x * torch.special.erfc(-x / 2**0.5) / 2
    far = x < -5.7
    assert far.sum() > 60
    assert ((y[:, far] - ref[far]).abs() <= ref[far].abs() * (0.0289 + 1e-4 + 2.0**-8)).all()
