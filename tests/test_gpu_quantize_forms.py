"""GPU checks of sp24_quantize_rows in the kernels that whole weights and batches of tokens take: a warp per row (592 rows and
more, up to 6144 entries, in four register widths) and a block per row (longer rows, or few), masked and not, in both types.
Bit for bit against the IEEE fp32 operations of the definition."""
import numpy as np
import pytest
import torch

import oracle
import structured_sparse_transformer_b200 as sp
from test_gpu_quantize import _reference

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _matrix(R, C, dt, seed):
    """Rows of unequal size, and among them rows of zeros, of one entry, with what is not finite, and of the smallest and
    largest numbers."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, C, generator=g) * torch.exp(0.5 * torch.randn(R, 1, generator=g))
    x = x.to(dt)
    for r in (3, R - 2):
        x[r] = 0
    x[5] = 0
    x[5, C // 2] = -1.5
    x[7, C - 1], x[9, 0], x[R - 5, C // 3] = float("nan"), float("inf"), -float("inf")
    x[11] = torch.finfo(dt).tiny
    x[12] = torch.finfo(dt).max
    x[13, C // 4] = 127.0
    x[13, C // 4 + 1:C // 4 + 9] = torch.arange(8) + 0.5
    return x


def _check(x, idx=None, pitch=0):
    R, C = x.shape
    base = torch.full((R, C + pitch), float("nan"), dtype=x.dtype, device="cuda")
    base[:, :C] = x.cuda()
    q = torch.full((R + 1, C), 77, dtype=torch.int8, device="cuda")
    s = torch.full((R + 1,), -5.0, device="cuda")
    sp.sp24_quantize_rows(base[:, :C], q, s, None if idx is None else torch.from_numpy(idx).cuda())
    torch.cuda.synchronize()
    assert (q[R:] == 77).all() and (s[R:] == -5.0).all()      # nothing behind the last row
    qr, sr = _reference(x, None if idx is None else oracle.dense_mask(idx).astype(bool))
    got, nan = s[:R].cpu().numpy(), np.isnan(sr)
    assert np.array_equal(np.isnan(got), nan)
    assert np.array_equal(got[~nan].view(np.uint32), sr[~nan].view(np.uint32))
    assert np.array_equal(q[:R].cpu().numpy(), qr)


# columns: up to 1024, 2048, 4096 and 6144 a warp per row in 4, 8, 16 and 24 units a lane; then a block per row
COLS = [64, 1000, 1024, 1032, 1600, 2048, 2056, 4000, 4096, 4104, 6000, 6144, 6152, 8192, 8200]


@pytest.mark.parametrize("C", COLS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_many_rows(C, dtype):
    _check(_matrix(592 + C % 13, C, DT[dtype], C))


@pytest.mark.parametrize("C", COLS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_many_rows_of_a_masked_weight(C, dtype):
    _masked(596 + 4 * (C % 3), C, dtype)


@pytest.mark.parametrize("C", [24, 2040, 2048, 2056, 4096, 6400, 8192, 8200])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_few_rows_of_a_masked_weight(C, dtype):
    _masked(20, C, dtype)


def _masked(R, C, dtype):
    x = _matrix(R, C, DT[dtype], C + 1)
    idx = np.random.default_rng(C).integers(0, 90, (R // 4, C // 4)).astype(np.uint8)
    keep = torch.from_numpy(oracle.dense_mask(idx).astype(bool))
    junk = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(x.dtype).max]).to(x.dtype)
    fill = junk[torch.randint(0, 4, (R, C), generator=torch.Generator().manual_seed(C))]
    x = torch.where(keep, x, fill)       # what a pruned place holds does not matter
    assert not torch.isfinite(x[:, :4]).all() and (~keep).any(1).all()
    _check(x, idx)


@pytest.mark.parametrize("C,pitch", [(1000, 8), (1600, 24), (4000, 96), (6000, 8), (1600, 1), (1000, 4)])
def test_many_pitched_rows(C, pitch):
    """A pitch of whole 16-byte units keeps the warp per row; another takes the form for any pitch."""
    _check(_matrix(601, C, torch.bfloat16, C + pitch), pitch=pitch)
