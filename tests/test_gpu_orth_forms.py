"""GPU checks of the orthogonalisation's forms (a grid over all matrices, a cluster per matrix, short sides up to 256) over the
numbers of rounds, in captured graphs and where the start's guess does not serve.  Tolerances as in test_gpu_orth.py."""
import pytest
import torch

import structured_sparse_transformer_b200 as sp
from test_gpu_orth import _grad, _ns, _orth, _rel, _tol, _workspace

pytestmark = pytest.mark.gpu


def _late(steps, m):
    """What rounds beyond the fifth add to the tolerance.  On a singular value a round is f(x) = a x + b x^3 + c x^5, and in
    the band 0.68..1.13 where values end f'(x) = a + 3 b x^2 + 5 c x^4 reaches -1.61 (at x^2 = -3 b / 10 c) and 1.72 (at
    1.13): f has no stable fixed point there.  What the roundings of a round move a value by (G's, P's and X's in fp16: a
    random matrix of relative entries 2^-11 / sqrt 3 has a spectral norm of at most 2 / sqrt 3 2^-11; 2^-10 for all three)
    can grow by 1.72 in each later round, up to the band's width of 0.45, and an emulation whose sums are rounded
    elsewhere is then at another place of the band.  One of m values there is 0.45 / (0.68 sqrt m) of the whole.
    (Seen at 512 x 512 after 16 rounds: of two matrices with a value on such a path, the emulation is 8.9e-3 and 1.7e-2
    off, the kernel 1.7e-2 and 5.5e-3; with sums in fp64 of the same rounded operands both stay within 8e-4 of one
    another for the first five rounds.)"""
    moved = 2.0**-10 * sum(1.72**r for r in range(max(steps - 5, 0)))
    return min(moved, 0.45) / (0.68 * m**0.5)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 7, 16])
@pytest.mark.parametrize("shape", [(777, 1333), (1333, 777), (300, 2000), (8, 512, 512), (4, 520, 300), (3, 96, 200), (200, 96)])
def test_rounds_in_every_form(shape, steps):
    """Even numbers end in the other buffer of X; one round is two phases with the norm's factor in the last product."""
    g = _grad(shape, steps + sum(shape))
    got = _orth(g, torch.float16, steps=steps)
    for z, x in zip(got.view(-1, *shape[-2:]), g.view(-1, *shape[-2:])):
        err, tol = _rel(z, _ns(x, steps)), _tol(x, torch.float16, steps) + _late(steps, min(x.shape))
        assert err <= tol, f"{shape} {steps}: {err:.2e} > {tol:.2e}"


@pytest.mark.parametrize("shape", [(700, 900), (1100, 520), (640, 1920), (4, 520, 300)])
def test_graphs_of_large_steps_equal_eager_ones(shape):
    """The grid over all matrices is a cooperative launch; captured and replayed it gives the eager step's bits."""
    g, m, w = _grad(shape, 1), _grad(shape, 2, 5e-3), _grad(shape, 3, 0.02)
    em, ew = m.clone(), w.clone()
    w16, e16 = (torch.empty(*shape, dtype=torch.float16, device="cuda") for _ in range(2))
    ws, es = _workspace(g), _workspace(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sp.sp24_muon_step(g, m, w, w16, ws, lr=0.01, weight_decay=0.1)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        sp.sp24_muon_step(g, em, ew, e16, es, lr=0.01, weight_decay=0.1)
    torch.cuda.synchronize()
    assert sp.sp24_device_status() == 0
    assert torch.equal(m, em) and torch.equal(w, ew) and torch.equal(w16, e16)


def test_two_graphs_of_large_matrices_side_by_side():
    gs = [_grad((700, 900), 1), _grad((520, 1100), 2)]
    want = [_orth(g) for g in gs]
    outs = [torch.empty(g.shape, dtype=torch.float16, device="cuda") for g in gs]
    spaces = [_workspace(g) for g in gs]
    graphs = [torch.cuda.CUDAGraph() for _ in gs]
    for gr, g, o, ws in zip(graphs, gs, outs, spaces):
        with torch.cuda.graph(gr):
            sp.sp24_orthogonalize(g, o, ws)
    streams = [torch.cuda.Stream() for _ in gs]
    torch.cuda.synchronize()
    for _ in range(4):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert sp.sp24_device_status() == 0
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@pytest.mark.parametrize("shape", [(96, 200), (200, 96), (3, 61, 130), (700, 900)])
@pytest.mark.parametrize("nesterov", [True, False])
def test_a_gradient_and_a_momentum_that_cancel(shape, nesterov):
    """U a thousandth of the gradient, from whose size the start's power of two is guessed: the start is rewritten.  The
    kernel forms m and U with one fused operation each, so U is the rounded value of g + mu m on the m that it returns."""
    mu = torch.tensor(0.95, dtype=torch.float32).double().item()
    g = _grad(shape, 1)
    r = torch.rand(shape, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")
    m0 = (g.double() * -((1 + mu) / mu**2 if nesterov else 1 / mu) * 1.001 * (1 + 1e-4 * r)).float()
    m, w = m0.clone(), _grad(shape, 3, 0.02)
    w0 = w.clone()
    sp.sp24_muon_step(g, m, w, None, _workspace(g), lr=0.05, nesterov=nesterov)
    torch.cuda.synchronize()
    assert sp.sp24_device_status() == 0
    exact = mu * m0.double() + g.double()
    assert ((m.double() - exact).abs() <= 2.0**-24 * exact.abs()).all()
    u = (g.double() + mu * m.double()).float() if nesterov else m
    assert u.norm() < 4e-3 * g.norm()
    u3 = u if u.dim() == 3 else u[None]
    o = torch.stack([_ns(x) for x in u3]).view(u.shape)
    upd = (w0.double() - w.double()) / 0.05
    tol = max(_tol(x) for x in u3) + 2.0**-22 * (w0.double().norm() / (0.05 * o.norm())).item()
    assert _rel(upd, o) <= tol
