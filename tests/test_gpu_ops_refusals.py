"""Calls of the optimiser-step and 8-bit entry points that are refused on a device, before anything is launched: buffers
that share memory where a kernel would read what another of its blocks has written.  Nothing changes."""
import pytest
import torch

import structured_sparse_transformer_b200 as sp

pytestmark = pytest.mark.gpu


def _refused(call, *buffers):
    before = [b.clone() for b in buffers]
    torch.cuda.synchronize()
    with pytest.raises(sp.Sp24Error, match="INVALID_ARG"):
        call()
    torch.cuda.synchronize()
    for b, was in zip(buffers, before):
        assert torch.equal(b.view(torch.uint8), was.view(torch.uint8))


def _bytes(n, fill=None):
    g = torch.Generator(device="cuda").manual_seed(n)
    return torch.randint(0, 60, (n,), generator=g, device="cuda").to(torch.uint8)


R, C = 64, 48


@pytest.mark.parametrize("where", ["W", "momentum", "grad", "the end of W"])
def test_a_16_bit_weight_over_another_buffer(where):
    mem = _bytes(5 * 4 * R * C)
    part = lambda k: mem[4 * R * C * k:4 * R * C * (k + 1)].view(torch.float32).view(R, C)
    g, m, w = part(0), part(1), part(3)
    ws = torch.empty(sp.sp24_orthogonalize_size(R, C), dtype=torch.uint8, device="cuda")
    at = {"grad": 0, "momentum": 4 * R * C + 2 * C, "W": 3 * 4 * R * C, "the end of W": 4 * 4 * R * C - 16}[where]
    w16 = mem[at:at + 2 * R * C].view(torch.float16).view(R, C)
    _refused(lambda: sp.sp24_muon_step(g, m, w, w16, ws, lr=0.1), mem)


@pytest.mark.parametrize("k", range(4))
def test_a_workspace_over_another_buffer(k):
    n = sp.sp24_orthogonalize_size(R, C)
    mem = _bytes(n + 4 * R * C)
    ws = mem[:n]
    shared = lambda dt: mem[n - 16:n - 16 + R * C * dt.itemsize].view(dt).view(R, C)
    f32 = lambda: torch.ones(R, C, device="cuda")
    bufs = [f32(), f32(), f32(), torch.ones(R, C, dtype=torch.float16, device="cuda")]
    bufs[k] = shared(bufs[k].dtype)
    _refused(lambda: sp.sp24_muon_step(*bufs, ws, lr=0.1), mem, *bufs)
    if k == 0:
        _refused(lambda: sp.sp24_orthogonalize(bufs[0], bufs[3], ws), mem)
    if k == 3:
        _refused(lambda: sp.sp24_orthogonalize(bufs[0], bufs[3], ws), mem, bufs[0])


def test_a_result_over_its_operands():
    mem = _bytes(1 << 16)
    x = mem[:2 * R * C].view(torch.float16).view(R, C)
    q = torch.zeros(R, C, dtype=torch.int8, device="cuda")
    s = torch.zeros(R, device="cuda")
    idx = mem[8192:8192 + R * C // 16].view(R // 4, C // 4)
    inside = mem[:R * C].view(torch.int8).view(R, C)
    at_end = mem[2 * R * C - 16:3 * R * C - 16].view(torch.int8).view(R, C)
    for bad_q, bad_s in ((inside, s), (at_end, s), (mem[8208:8208 + R * C].view(torch.int8).view(R, C), s),
                         (q, mem[64:64 + 4 * R].view(torch.float32)), (q, mem[8192:8192 + 4 * R].view(torch.float32)),
                         (q, q.view(torch.uint8).view(-1)[:4 * R].view(torch.float32))):
        _refused(lambda: sp.sp24_quantize_rows(x, bad_q, bad_s, idx), mem, q, s)


@pytest.mark.parametrize("T", [1, 20, 64])
def test_a_product_over_its_operands(T):
    K, N = 64, 48
    mem = _bytes(1 << 16)
    xq, wq = mem[:T * K].view(torch.int8).view(T, K), mem[16384:16384 + N * K].view(torch.int8).view(N, K)
    sx, sw = mem[32768:32768 + 4 * T].view(torch.float32), mem[40960:40960 + 4 * N].view(torch.float32)
    y_at = lambda at: mem[at:at + 2 * T * N].view(torch.bfloat16).view(T, N)
    for at in (0, 16384 - 16, 32768, 40960):
        if at == 16384 - 16 and 2 * T * N <= 16:
            continue
        _refused(lambda: sp.sp24_gemm_i8(xq, sx, wq, sw, y_at(at)), mem)


def test_neighbouring_buffers_are_taken():
    """Side by side without a gap: nothing is shared."""
    mem = _bytes(1 << 16)
    x, q = mem[:2 * R * C].view(torch.float16).view(R, C), mem[2 * R * C:3 * R * C].view(torch.int8).view(R, C)
    s = mem[3 * R * C:3 * R * C + 4 * R].view(torch.float32)
    sp.sp24_quantize_rows(x, q, s)
    want_q, want_s = torch.empty(R, C, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    sp.sp24_quantize_rows(x.clone(), want_q, want_s)
    assert torch.equal(q, want_q) and torch.equal(s, want_s)
    n = sp.sp24_orthogonalize_size(R, C)
    both = torch.zeros(n + 6 * R * C, dtype=torch.uint8, device="cuda")
    g = both[n:n + 4 * R * C].view(torch.float32).view(R, C).normal_()
    out = both[n + 4 * R * C:].view(torch.float16).view(R, C)
    sp.sp24_orthogonalize(g, out, both[:n])
    want = torch.empty(R, C, dtype=torch.float16, device="cuda")
    sp.sp24_orthogonalize(g, want, both[:n])
    assert torch.equal(out, want)
