"""GPU checks of sp24_gemm_i8 against the definition in 64 bits.

Tolerance, per element: the integer sum is exact.  Its conversion to fp32 and the two products are off by
at most 2^-24 each, relative, so the pre-rounding value by 3 (2^-24)(1 + 2^-23); the store by eps/2 of the
dtype, or half a subnormal step (fp16 2^-25) near zero.  GELU = max(x, 0) - |x| t with t = erfc(|x|/sqrt 2)/2:
t comes from a polynomial within 9.1e-6, an exponential within 2^-22 whose argument (up to 2^6 before the
result falls under fp16's range) is off by 2 (2^-24) relative, i.e. t within 2.5e-5, and beyond |x| = 5.66, where the
polynomial's argument is clamped, |x| t is at most 4.4e-8; the input error passes through with gelu' (at most
1.13), and the last fused operation rounds by 2^-24."""
import numpy as np
import pytest
import torch

import structured_sparse_transformer_b200 as sp

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _operands(T, K, N, seed, full=False):
    g = torch.Generator().manual_seed(seed)
    lo = -128 if full else -127
    xq = torch.randint(lo, 128, (T, K), generator=g).to(torch.int8)
    wq = torch.randint(lo, 128, (N, K), generator=g).to(torch.int8)
    sx = torch.rand(T, generator=g) * 0.02 + 1e-3
    sw = (torch.rand(N, generator=g) + 0.05) / (73.0 * 73.0 * K**0.5 * 0.02)
    return xq, sx, wq, sw


def _reference(xq, sx, wq, sw):
    acc = xq.double() @ wq.double().t()          # exact: below 2^53
    return acc * sw.double() * sx.double()[:, None]


def _tolerance(x, ref, epi, dt):
    rel = 3 * 2.0**-24 * (1 + 2.0**-23)
    half = torch.finfo(dt).eps / 2
    sub = 2.0**-25 if dt == torch.float16 else 0.0
    if epi is None:
        before = x.abs() * rel
    else:
        t = torch.special.erfc(x.abs() / 2**0.5) / 2
        before = x.abs() * (t * 2.5e-5 + 1.13 * rel) + 4.4e-8 + 2.0**-24 * ref.abs()
    return before * (1 + half) + half * ref.abs() + sub


def _check(xq, sx, wq, sw, dtype, epi, stream=None):
    dt = DT[dtype]
    T, N = xq.shape[0], wq.shape[0]
    y = torch.full((T + 2, N), 7.0, dtype=dt, device="cuda")
    sp.sp24_gemm_i8(xq.cuda(), sx.cuda(), wq.cuda(), sw.cuda(), y, epi, stream=stream)
    torch.cuda.synchronize()
    assert sp.sp24_device_status() == 0
    assert (y[T:] == 7.0).all()                  # rows behind the last token are left as they were
    x = _reference(xq, sx, wq, sw)
    ref = x if epi is None else x * torch.special.ndtr(x)
    got = y[:T].cpu().double()
    assert torch.isfinite(got).all()
    worst = ((got - ref).abs() / _tolerance(x, ref, epi, dt).clamp_min(1e-300)).max().item()
    assert worst <= 1.0, f"T={T} {tuple(wq.shape)} {dtype} {epi}: {worst:.3f} of the tolerance"
    return y


SIZES = [(1, 16, 16), (1, 64, 256), (1, 1600, 6400), (2, 48, 80), (3, 5120, 1280), (4, 1024, 4096), (5, 656, 144), (8, 272, 528), (16, 2064, 400),
         (17, 128, 256), (31, 1600, 112), (32, 6400, 1600), (33, 144, 272), (37, 5120, 1280), (64, 256, 256), (65, 400, 272),
         (100, 96, 1040), (128, 1024, 4096), (129, 1040, 512), (255, 208, 304), (257, 512, 256), (700, 1024, 4096),
         (2047, 1024, 4096), (4096, 640, 2576)]


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("dtype,epi", [("f16", None), ("bf16", "gelu")])
def test_product(T, K, N, dtype, epi):
    _check(*_operands(T, K, N, T + K + N), dtype, epi)


@pytest.mark.parametrize("T", [1, 5, 40, 300])
@pytest.mark.parametrize("dtype,epi", [("f16", "gelu"), ("bf16", None)])
def test_product_other_types(T, dtype, epi):
    _check(*_operands(T, 1600, 272, T), dtype, epi)


@pytest.mark.parametrize("T", [1, 4, 20, 200])
def test_the_largest_sums_are_exact(T):
    """K at its limit with every product 128 * 128: 2^31 - 2^18 + ..., no overflow and no rounding of the sum."""
    K, N = 131056, 32
    xq = torch.full((T, K), -128, dtype=torch.int8)
    wq = torch.full((N, K), -128, dtype=torch.int8)
    wq[1] = 127
    wq[2] = 0
    wq[3, ::2] = 127
    sx, sw = torch.ones(T), torch.full((N,), 2.0**-17)
    y = _check(xq, sx, wq, sw, "bf16", None)
    assert float(y[0, 0]) == float(torch.tensor(K * 16384 * 2.0**-17).bfloat16())


def test_each_operand_entry_lands_where_it_should():
    """One nonzero entry at a time: k in every 16-byte unit of a stage, the first and the last row."""
    K, N = 400, 288
    for T in (1, 9, 200):
        xq, wq = torch.zeros(T, K, dtype=torch.int8), torch.zeros(N, K, dtype=torch.int8)
        for k in range(0, K, 13):
            xq[k % T, k] = (k % 120) + 1
            wq[(7 * k) % N, k] = -((3 * k) % 120) - 1
        _check(xq, torch.ones(T), wq, torch.full((N,), 2.0**-8), "f16", None)


@pytest.mark.parametrize("T", [1, 3, 40])
def test_scales_of_zero_and_nan(T):
    xq, sx, wq, sw = _operands(T, 320, 64, 9)
    sw[3] = 0.0
    sx[0] = float("nan")          # a token whose row was not finite
    y = torch.empty(T, 64, dtype=torch.float16, device="cuda")
    sp.sp24_gemm_i8(xq.cuda(), sx.cuda(), wq.cuda(), sw.cuda(), y)
    y = y.cpu()
    assert torch.isnan(y[0]).all() and not torch.isnan(y[1:]).any() and (y[1:, 3] == 0).all()


@pytest.mark.parametrize("T", [1, 3, 37, 600])
def test_results_do_not_depend_on_the_batch_and_repeat(T):
    xq, sx, wq, sw = [t.cuda() for t in _operands(T, 1600, 528, 11)]
    outs = []
    for _ in range(3):
        y = torch.empty(T, 528, dtype=torch.float16, device="cuda")
        sp.sp24_gemm_i8(xq, sx, wq, sw, y, "gelu")
        outs.append(y)
    one = torch.empty(1, 528, dtype=torch.float16, device="cuda")
    sp.sp24_gemm_i8(xq[T // 2:T // 2 + 1].contiguous(), sx[T // 2:T // 2 + 1].contiguous(), wq, sw, one, "gelu")
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert torch.equal(one[0], outs[0][T // 2])


def test_no_tokens_and_a_side_stream_and_a_graph():
    xq, sx, wq, sw = [t.cuda() for t in _operands(5, 640, 256, 4)]
    sp.sp24_gemm_i8(xq[:0], sx[:0], wq, sw, torch.empty(0, 256, dtype=torch.float16, device="cuda"))
    want = torch.empty(5, 256, dtype=torch.float16, device="cuda")
    sp.sp24_gemm_i8(xq, sx, wq, sw, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = torch.empty_like(want)
    sp.sp24_gemm_i8(xq, sx, wq, sw, got, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    got.zero_()
    with torch.cuda.graph(g):
        sp.sp24_gemm_i8(xq, sx, wq, sw, got)
    for k in range(2):
        xq.neg_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, -want if k == 0 else want)


def test_quantized_layer_stays_near_the_16_bit_one():
    """x W^T through quantize + product: each factor off by at most half a step of its row, so by Cauchy-Schwarz
    |error| <= (sx |w|_1 + sw |x|_1) / 2 + K sx sw / 4."""
    T, K, N = 50, 1600, 400
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(T, K, generator=g).half(), (torch.randn(N, K, generator=g) * 0.02).half()
    q = []
    for m in (x, w):
        a, s = torch.empty(m.shape, dtype=torch.int8, device="cuda"), torch.empty(m.shape[0], device="cuda")
        sp.sp24_quantize_rows(m.cuda(), a, s)
        q.append((a, s))
    y = torch.empty(T, N, dtype=torch.float16, device="cuda")
    sp.sp24_gemm_i8(q[0][0], q[0][1], q[1][0], q[1][1], y)
    ref = x.double() @ w.double().t()
    sx, sw = q[0][1].cpu().double()[:, None] * (1 + 2.0**-14), q[1][1].cpu().double() * (1 + 2.0**-14)
    bound = 0.5 * (sx * w.double().abs().sum(1) + sw * x.double().abs().sum(1, keepdim=True)) + 0.25 * K * sx * sw
    bound = bound + ref.abs() * 2.0**-10
    assert ((y.cpu().double() - ref).abs() <= bound).all()


def test_an_expired_wait_is_reported_and_the_next_call_is_right():
    # (K long enough that no wait is over before it starts: 65536 in 64 or more steps)
    for T, K in ((40, 65536), (3000, 65536)):
        xq, sx, wq, sw = [t.cuda() for t in _operands(T, K, 528, 2)]
        want, y = (torch.empty(T, 528, dtype=torch.float16, device="cuda") for _ in range(2))
        sp.sp24_gemm_i8(xq, sx, wq, sw, want)
        try:
            sp.sp24_set_wait_budget(0)
            sp.sp24_gemm_i8(xq, sx, wq, sw, y)
            torch.cuda.synchronize()
        finally:
            sp.sp24_set_wait_budget(1 << 32)
        assert sp.sp24_device_status() == 6
        sp.sp24_gemm_i8(xq, sx, wq, sw, y)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and sp.sp24_device_status() == 0


def test_outputs_past_32_bit_offsets():
    """T N beyond 2^31 elements (5.4 GB): the last tokens are as in a small call, what lies behind is untouched."""
    T, K, N = 40961, 64, 65552
    g = torch.Generator(device="cuda").manual_seed(5)
    xq = torch.randint(-127, 128, (T, K), generator=g, device="cuda").to(torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda").to(torch.int8)
    sx = torch.rand(T, generator=g, device="cuda") * 0.01
    sw = torch.rand(N, generator=g, device="cuda") * 0.01
    y = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    sp.sp24_gemm_i8(xq, sx, wq, sw, y)
    for lo, hi in ((0, 3), (T // 2, T // 2 + 3), (T - 3, T)):
        part = torch.empty(hi - lo, N, dtype=torch.bfloat16, device="cuda")
        sp.sp24_gemm_i8(xq[lo:hi].contiguous(), sx[lo:hi].contiguous(), wq, sw, part)
        assert torch.equal(y[lo:hi], part)
    assert (y[T:] == 7.0).all() and sp.sp24_device_status() == 0


@pytest.mark.parametrize("K,N", [(6400, 640), (4000, 1600), (3200, 3216), (9600, 6400)])
@pytest.mark.parametrize("T", [1, 2, 3, 8, 12, 30, 60, 120, 300])
def test_long_contractions_of_few_tokens(T, K, N):
    """K in eight to one parts, every token tile; the last parts of K are shorter."""
    _check(*_operands(T, K, N, T + K), "bf16", None)


@pytest.mark.parametrize("K", [16, 2048, 2064, 6400])
@pytest.mark.parametrize("T", [1, 2, 4, 5])
def test_dot_products_of_odd_lengths(T, K):
    """Units of 16 that end anywhere in a thread's turn."""
    _check(*_operands(T, K, 400, T + K, full=True), "f16", "gelu")
