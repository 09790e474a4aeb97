"""GPU checks of sp24_orthogonalize and sp24_muon_step against the iteration in 64 bits.

Tolerance (relative Frobenius).  The kernels round the iterate, the Gram matrix and the polynomial to fp16
(half a step 2^-11) once a round each and accumulate in fp32.  An emulation in fp64 that rounds at the same
places gives the error e of these roundings for the same input; the kernel's own differ from it only where
fp32 accumulation moves a value across a rounding border, so its error is of the same size: 2 e is allowed,
or 8 (2^-11) where a matrix is so small that e is one draw of few roundings (15 of them, each 2^-11/sqrt 3
with a gain of about 2: 4.5 (2^-11) as a standard deviation); then eps/2 of the output type."""
import math

import numpy as np
import pytest
import torch

import oracle
import structured_sparse_transformer_b200 as sp
import synthetic_inputs as si

pytestmark = pytest.mark.gpu
A, B, C = 3.4445, -4.7750, 2.0315
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _ns(g, steps=5, eps=1e-7, half=False):
    """The iteration in fp64 on one matrix (on the GPU); half: with the kernels' roundings."""
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    rnd = (lambda v: v.half().double()) if half else (lambda v: v)
    s = 2.0 ** math.floor(math.log2(max(x.shape)) / 2)
    x = rnd(x / (x.norm() + eps) * s)
    eye = torch.eye(x.shape[0], dtype=x.dtype, device=x.device)
    for k in range(steps):
        a = rnd(x @ x.t() / s**2)
        x = rnd(A * eye + B * a + C * (a @ a)) @ x
        x = rnd(x) if k + 1 < steps else x
    x = x / s
    return x.t() if tall else x


def _rel(a, b):
    return ((a.double() - b).norm() / b.norm().clamp_min(1e-300)).item()


def _tol(g, dt=None, steps=5, eps=1e-7):
    e = _rel(_ns(g, steps, eps, half=True), _ns(g, steps, eps))
    return max(2 * e, 8 * 2.0**-11) + (torch.finfo(dt).eps / 2 if dt is not None else 0.0)


def _grad(shape, seed, std=1e-3):
    g = torch.Generator().manual_seed(seed)
    m = torch.randn(*shape, generator=g) * torch.exp(0.5 * torch.randn(*shape[:-2], 1, shape[-1], generator=g))
    m = m + torch.randn(*shape[:-1], 4, generator=g) @ torch.randn(*shape[:-2], 4, shape[-1], generator=g)
    return (m * std).cuda()


def _workspace(g):
    c, r, k = (1, *g.shape) if g.dim() == 2 else g.shape
    # its contents do not matter: every call gets one full of NaN patterns
    return torch.full((sp.sp24_orthogonalize_size(r, k, c),), 0xFF, dtype=torch.uint8, device="cuda")


def _orth(g, dt=torch.float16, **kw):
    out = torch.full((g.numel() + 8,), 7.0, dtype=dt, device="cuda")
    sp.sp24_orthogonalize(g, out, _workspace(g), **kw)
    torch.cuda.synchronize()
    assert sp.sp24_device_status() == 0
    assert (out[g.numel():] == 7.0).all()
    return out[:g.numel()].view(g.shape)


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 2), (3, 130), (16, 16), (64, 64), (65, 63), (127, 129), (128, 256), (130, 67),
          (256, 512), (257, 255), (300, 1000), (512, 256), (777, 1333), (1333, 777), (1000, 40), (8, 4096), (1280, 5120)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_orthogonalize(shape, dtype):
    g = _grad(shape, sum(shape))
    got = _orth(g, DT[dtype])
    err, tol = _rel(got, _ns(g)), _tol(g, DT[dtype])
    assert err <= tol, f"{shape} {dtype}: {err:.2e} > {tol:.2e}"


@pytest.mark.parametrize("steps", [1, 2, 3, 6, 10])
def test_steps(steps):
    g = _grad((96, 200), steps)
    err, tol = _rel(_orth(g, steps=steps), _ns(g, steps)), _tol(g, torch.float16, steps)
    assert err <= tol, f"{err:.2e} > {tol:.2e}"


def test_singular_values_end_near_one():
    g = _grad((320, 640), 5)
    s = torch.linalg.svdvals(_orth(g, torch.bfloat16).double())
    assert 0.6 < s.min() and s.max() < 1.25


@pytest.mark.parametrize("count,shape", [(2, (64, 96)), (3, (451, 317)), (5, (33, 129)), (7, (260, 8)), (8, (512, 512))])
def test_stack_equals_its_matrices(count, shape):
    g = _grad((count, *shape), count)
    whole = _orth(g, torch.bfloat16)
    for k in range(count):
        one = _orth(g[k].contiguous(), torch.bfloat16)
        err, tol = _rel(whole[k], _ns(g[k])), _tol(g[k], torch.bfloat16)
        assert err <= tol
        # the norm's partial sums may be grouped otherwise, nothing else
        assert _rel(whole[k], one.double()) <= tol
    assert torch.equal(whole, _orth(g, torch.bfloat16))


def test_pitched_rows_and_spaced_matrices():
    big = _grad((3, 70, 100), 8)
    view = big[:, 5:66, 3:90]                       # pitch 100, matrices 7000 apart, rows not 16-byte aligned
    base = torch.zeros(3, 61, 100, device="cuda")
    base[:, :, :87] = view
    got = _orth(base[:, :, :87])
    assert torch.equal(got, _orth(base[:, :, :87].contiguous()))
    assert torch.equal(got, _orth(view))


@pytest.mark.parametrize("shape", [(60, 44), (44, 60), (45, 61)])
def test_buffers_at_odd_addresses(shape):
    """fp32 buffers 4 bytes and 16-bit buffers 2 bytes past a 16-byte boundary."""
    n = shape[0] * shape[1]
    at = lambda t, k: torch.empty(n + 8, dtype=t.dtype, device="cuda")[k:k + n].view(shape).copy_(t)
    g, m, w = _grad(shape, 1), _grad(shape, 2), _grad(shape, 3, 0.02)
    want = _orth(g)
    for k in (1, 2, 4):
        got = at(torch.zeros_like(want), k)
        sp.sp24_orthogonalize(at(g, k), got, _workspace(g))
        assert _rel(got, want.double()) <= _tol(g, torch.float16)
        m1, w1, h1 = at(m, k), at(w, k), at(want, k)
        m0, w0, h0 = m.clone(), w.clone(), want.clone()
        sp.sp24_muon_step(at(g, k), m1, w1, h1, _workspace(g), lr=0.1)
        sp.sp24_muon_step(g, m0, w0, h0, _workspace(g), lr=0.1)
        assert torch.equal(m0, m1) and torch.equal(h1, w1.half())
        assert (w1 - w0).norm() <= 0.1 * 8 * 2.0**-11 * min(shape) ** 0.5


def test_scale_of_the_input_does_not_matter():
    g = _grad((200, 300), 4, std=1.0)
    want = _ns(g, eps=0.0)
    for f in (1e-30, 1e-18, 1e-3, 1e10, 1e25, 1e33):
        got = _orth(g * f, eps=0.0)
        assert _rel(got, want) <= _tol(g, torch.float16, eps=0.0), f
    # eps counts: |G| = eps halves the first iterate
    h = g / g.norm() * 1e-3
    assert _rel(_orth(h, eps=1e-3, steps=1), _ns(h, 1, 1e-3)) <= _tol(h, torch.float16, 1, 1e-3)


def test_matrices_of_nothing_and_of_one_entry():
    z = torch.zeros(2, 40, 30, device="cuda")
    z[1, 3, 4] = -2.0
    got = _orth(z, eps=0.0)
    assert (got[0] == 0).all()
    ref = _ns(z[1], eps=0.0)
    assert abs(got[1, 3, 4].item() - ref[3, 4].item()) <= _tol(z[1], torch.float16) and int((got[1] != 0).sum()) == 1
    sp.sp24_orthogonalize(torch.zeros(0, 5, device="cuda"), torch.zeros(0, 5, dtype=torch.float16, device="cuda"),
                          torch.zeros(0, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_stays_in_its_matrix(junk):
    g = _grad((3, 50, 70), 6)
    clean = _orth(g)
    g[1, 7, 9] = junk
    got = _orth(g)
    assert torch.isnan(got[1]).all() and torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])


def _muon_reference(g, m, w, mu, nesterov, lr, wd, scale, steps=5):
    m = mu * m.double() + g.double()
    u = g.double() + mu * m if nesterov else m
    u3 = u if u.dim() == 3 else u[None]
    o = torch.stack([_ns(x, steps) for x in u3]).view(u.shape)
    return m, u, o, (1 - lr * wd) * w.double() - lr * scale * o


@pytest.mark.parametrize("shape", [(1, 1), (1, 9), (64, 96), (96, 64), (129, 77), (77, 129), (512, 256), (3, 100, 44),
                                   (2, 44, 101), (4, 256, 384), (6400, 1600)])
@pytest.mark.parametrize("dtype,nesterov", [("f16", True), ("bf16", False)])
def test_muon_step(shape, dtype, nesterov):
    dt = DT[dtype]
    lr, wd, mu, scale = 0.03, 0.1, 0.95, 0.7
    g, m = _grad(shape, 1), _grad(shape, 2, 5e-3)
    w = (torch.randn(*shape, generator=torch.Generator().manual_seed(3)) * 0.02).cuda()
    w0, g0 = w.clone(), g.clone()
    rm, u, o, rw = _muon_reference(g, m, w, mu, nesterov, lr, wd, scale)
    w16 = torch.empty(*shape, dtype=dt, device="cuda")
    sp.sp24_muon_step(g, m, w, w16, _workspace(g), lr=lr, mu=mu, nesterov=nesterov, weight_decay=wd, scale=scale)
    torch.cuda.synchronize()
    assert sp.sp24_device_status() == 0
    assert torch.equal(g, g0)
    # mu is passed as fp32 (half a step 2^-24 off), then one fused operation: 2 half steps of each part
    assert ((m.double() - rm).abs() <= 2.0**-23 * (rm.abs() + (rm - g.double()).abs())).all()
    assert torch.equal(w16, w.to(dt))
    # the update alone: W's own rounding (half a step of |keep W| and of W, and of lr wd) over the step's size
    upd = ((1 - lr * wd) * w0.double() - w.double()) / (lr * scale)
    u3 = u if u.dim() == 3 else u[None]
    tol = max(_tol(x) for x in u3) + 2.0**-22 * (w0.double().norm() / (lr * scale * o.norm())).item()
    err = _rel(upd, o)
    assert err <= tol, f"{err:.2e} > {tol:.2e}"


def test_muon_without_a_16_bit_copy_and_without_decay():
    g, m, w = _grad((80, 48), 1), _grad((80, 48), 2), _grad((80, 48), 3, 0.02)
    a = [t.clone() for t in (m, w)]
    w16 = torch.empty(80, 48, dtype=torch.float16, device="cuda")
    sp.sp24_muon_step(g, m, w, None, _workspace(g), lr=0.02)
    sp.sp24_muon_step(g, a[0], a[1], w16, _workspace(g), lr=0.02)
    assert torch.equal(m, a[0]) and torch.equal(w, a[1])


def test_graph_replays_equal_eager_steps_on_a_side_stream():
    shape = (2, 96, 160)
    g, m, w = _grad(shape, 1), _grad(shape, 2), _grad(shape, 3, 0.02)
    em, ew = m.clone(), w.clone()
    w16, e16 = (torch.empty(*shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws, es = _workspace(g), _workspace(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sp.sp24_muon_step(g, m, w, w16, ws, lr=0.01, weight_decay=0.1)
    side = torch.cuda.Stream()
    for _ in range(3):
        graph.replay()
        sp.sp24_muon_step(g, em, ew, e16, es, lr=0.01, weight_decay=0.1, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(m, em) and torch.equal(w, ew) and torch.equal(w16, e16)


def test_two_streams_at_once():
    """Independent calls side by side, each with its workspace: large (one cooperative grid each) and small ones."""
    shapes = [(640, 1920), (1100, 520), (256, 512), (2, 64, 96)]
    gs = [_grad(s, k) for k, s in enumerate(shapes)]
    want = [_orth(g) for g in gs]
    streams = [torch.cuda.Stream() for _ in shapes]
    outs = [torch.empty(g.shape, dtype=torch.float16, device="cuda") for g in gs]
    spaces = [_workspace(g) for g in gs]
    torch.cuda.synchronize()
    for _ in range(4):
        for g, o, w, st in zip(gs, outs, spaces, streams):
            sp.sp24_orthogonalize(g, o, w, stream=st)
    torch.cuda.synchronize()
    assert sp.sp24_device_status() == 0
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


def test_two_graphs_with_their_own_workspaces():
    g = _grad((130, 200), 3)
    want = _orth(g)
    graphs, outs, spaces = [], [], []
    for _ in range(2):
        out, ws = torch.empty(130, 200, dtype=torch.float16, device="cuda"), _workspace(g)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            sp.sp24_orthogonalize(g, out, ws)
        graphs.append(gr)
        outs.append(out)
        spaces.append(ws)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want) and sp.sp24_device_status() == 0


def test_an_expired_wait_is_reported_and_the_next_call_is_right():
    for shape in ((700, 900), (64, 96)):       # a grid, a cluster
        g = _grad(shape, 2)
        want = _orth(g)
        try:
            sp.sp24_set_wait_budget(0)
            sp.sp24_orthogonalize(g, torch.empty(*shape, dtype=torch.float16, device="cuda"), _workspace(g), steps=2)
            torch.cuda.synchronize()
        finally:
            sp.sp24_set_wait_budget(1 << 32)
        assert sp.sp24_device_status() == 6
        assert torch.equal(_orth(g), want)


def test_from_the_gradient_to_the_8_bit_layer():
    """A training step's end and an 8-bit evaluation of it: Muon step of both weights on masked gradients, mask step,
    quantisation of the masked weights, two products with a GELU and a quantisation between them.  Each stage is
    checked against its definition on the stage's own inputs."""
    d, ff, T = 128, 320, 50
    x = si.normal((T, d), 1.0, 1, "f16").cuda()
    weights = []
    for k, (r, c) in enumerate(((ff, d), (d, ff))):
        w = (torch.randn(r, c, generator=torch.Generator().manual_seed(k)) * 0.02).cuda()
        w16 = w.half()
        idx = torch.empty(r // 4, c // 4, dtype=torch.uint8, device="cuda")
        sp.sp24_mask_search(w16, idx)
        grad, mom = _grad((r, c), 10 + k), torch.zeros(r, c, device="cuda")
        sp.sp24_masked_decay(grad, w16, idx, 1e-3)
        _, u, o, rw = _muon_reference(grad, mom, w, 0.95, True, 0.02, 0.1, 1.0)
        sp.sp24_muon_step(grad, mom, w, w16, _workspace(grad), lr=0.02, weight_decay=0.1)
        tol = 0.02 * _tol(u) * o.norm().item() + 2.0**-22 * rw.norm().item()
        assert (w.double() - rw).norm().item() <= tol
        new = torch.empty_like(idx)
        flips = torch.zeros(1, dtype=torch.int64, device="cuda")
        sp.sp24_mask_step(w16, new, idx, flips)
        ref_idx = oracle.mask_search(si.bits16(w16.cpu()), "f16")
        assert np.array_equal(new.cpu().numpy(), ref_idx) and int(flips) == oracle.flip_count(idx.cpu().numpy(), ref_idx)
        q, s = torch.empty(r, c, dtype=torch.int8, device="cuda"), torch.empty(r, device="cuda")
        sp.sp24_quantize_rows(w16, q, s, new)
        keep = torch.from_numpy(oracle.dense_mask(ref_idx).astype(bool)).cuda()
        assert (q[~keep] == 0).all()
        step = (q.double() * s.double()[:, None] - torch.where(keep, w16, torch.zeros_like(w16)).double()).abs()
        assert (step <= s.double()[:, None] * (0.5 + 2.0**-14)).all()
        weights.append((q, s))
    a = x
    for k, epi in enumerate(("gelu", None)):
        qa, sa = torch.empty(a.shape, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        sp.sp24_quantize_rows(a, qa, sa)
        q, s = weights[k]
        y = torch.empty(T, q.shape[0], dtype=torch.float16, device="cuda")
        sp.sp24_gemm_i8(qa, sa, q, s, y, epi)
        z = (qa.double() @ q.double().t()) * s.double() * sa.double()[:, None]
        ref = z * torch.special.ndtr(z) if epi else z
        assert ((y.double() - ref).abs() <= 2.0**-11 * ref.abs() + z.abs() * 1.5e-5 + 2.0**-25 + 4.4e-8).all()
        a = y
    assert sp.sp24_device_status() == 0


@pytest.mark.parametrize("shape", [(96, 200), (200, 96), (3, 61, 130)])
@pytest.mark.parametrize("case", ["zero gradient", "tiny gradient", "momentum of the other sign", "a huge entry",
                                  "zeros where sizes are guessed"])
def test_starts_of_unusual_sizes(shape, case):
    """The first fp16 iterate's power of two is guessed from the gradient at some places; where the guess does not
    serve, the result is the same."""
    g, m = _grad(shape, 1), _grad(shape, 2, 5e-3)
    if case == "zero gradient":
        g.zero_()
    elif case == "tiny gradient":
        g *= 1e-20
    elif case == "momentum of the other sign":
        m = -g / 0.95 * (1 + 1e-6)
    elif case == "a huge entry":
        g.view(-1)[g.numel() // 3 + 1] = 3e4
    else:
        n = shape[-1] * shape[-2]
        at = (n // 8 * torch.arange(8)[:, None] + torch.arange(32)).flatten().clamp_max(n - 1).cuda()
        g.view(-1, n)[:, at] = 0.0
    w = _grad(shape, 3, 0.02)
    w0 = w.clone()
    _, u, o, _ = _muon_reference(g, m, w, 0.95, True, 0.05, 0.0, 1.0)
    sp.sp24_muon_step(g, m, w, None, _workspace(g), lr=0.05)
    if case == "momentum of the other sign":     # what cancels in U is rounded to 32 bits there: take U's own value
        u = g.double() + 0.95 * m.double()
        u = u.float()
        o = torch.stack([_ns(x) for x in (u if u.dim() == 3 else u[None])]).view(u.shape)
    u3 = u if u.dim() == 3 else u[None]
    upd = (w0.double() - w.double()) / 0.05
    tol = max(_tol(x) for x in u3) + 2.0**-22 * (w0.double().norm() / (0.05 * o.norm())).item()
    if case == "momentum of the other sign":     # (the fp32 sum of U: half a step of |g| + |mu m|, over |U|; the
        tol = tol + 3.4445**5 * (2.0**-23 * 2 * g.double().norm() / u.double().norm()).item()   # rounds raise small parts a^5 times)
    assert _rel(upd, o) <= tol
    one = torch.empty(*shape, dtype=torch.float16, device="cuda")
    sp.sp24_orthogonalize(u.float().contiguous(), one, _workspace(g), steps=1)
    ref = torch.stack([_ns(x.float(), 1) for x in u3]).view(u.shape)
    assert _rel(one, ref) <= max(_tol(x.float(), torch.float16, 1) for x in u3)


def test_momentum_that_shares_memory_is_refused():
    g, w = _grad((64, 48), 1), _grad((64, 48), 2, 0.02)
    ws = _workspace(g)
    w0, g0 = w.clone(), g.clone()
    both = torch.zeros(100, 48, device="cuda")
    for args in ((g, g, w), (g, w, w)):
        with pytest.raises(ValueError, match="momentum"):
            sp.sp24_muon_step(*args, None, ws, lr=0.1)
    with pytest.raises(RuntimeError, match="INVALID_ARG"):   # rows in common
        sp.sp24_muon_step(both[:64], both[36:], w, None, ws, lr=0.1)
    torch.cuda.synchronize()
    assert torch.equal(w, w0) and torch.equal(g, g0) and not both.any()
