"""Cases of the library's optimiser-step and 8-bit operators, for timing and for comparison.

Five calls of the binding are covered:

- ``sp24_orthogonalize``: a weight-shaped matrix G becomes O = NS(G / (|G|_F + eps)), NS being `steps` rounds of
  X <- a X + (b A + c A^2) X with A = X X^T (the quintic Newton-Schulz iteration of the Muon optimiser).
- ``sp24_muon_step``: momentum, orthogonalisation and weight update in one call, on the fp32 master weight, the
  momentum and the 16-bit weight that the mask search and the products read.
- ``sp24_quantize_rows``: rows of a 16-bit matrix (tokens, or output channels of a masked weight) to 8-bit integers
  and a scale a row.
- ``sp24_gemm_i8``: the product of 8-bit activations and weights with a scale for each token and channel, alone or
  behind a GELU.

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the library's calls.
"""
import itertools
import math

import torch

own = False

A, B, C = 3.4445, -4.7750, 2.0315      # the quintic's coefficients
EPS = 1e-7
STEPS = 5
MU = 0.95
WEIGHT_DECAY = 0.1
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one weight of the smoke check's layer: launch latency counts
        dict(name="muon-small", op="muon", count=1, rows=512, cols=256, dtype="f16", nesterov=True, lr=5e-5),
        # the up projection of GPT-2 1.5B alone, as in a step that goes weight by weight
        dict(name="muon-1p5b-w1", op="muon", count=1, rows=6400, cols=1600, dtype="f16", nesterov=True, lr=5e-5),
        # the up projections of eight layers of GPT-2 355M, stacked
        dict(name="muon-355m-stack", op="muon", count=8, rows=4096, cols=1024, dtype="f16", nesterov=True, lr=5e-5),
        # odd sizes, rows of no round pitch, heavy-ball momentum
        dict(name="muon-ragged", op="muon", count=1, rows=777, cols=1333, dtype="bf16", nesterov=False, lr=5e-5),
        # the down projection of GPT-2 774M: the orthogonalisation alone, for a program with its own momentum
        dict(name="orth-774m-w2", op="orth", count=1, rows=1280, cols=5120, dtype="bf16"),
        # a few small projections with odd sides, stacked
        dict(name="orth-ragged-stack", op="orth", count=3, rows=451, cols=317, dtype="bf16"),
        # hidden activations of GPT-2 774M before the down projection
        dict(name="quant-hidden", op="quant", rows=16384, cols=5120, dtype="bf16", masked=False),
        # the masked up projection of GPT-2 1.5B, once after training
        dict(name="quant-w1-masked", op="quant", rows=6400, cols=1600, dtype="f16", masked=True),
        # one token through the up projection of GPT-2 1.5B
        dict(name="i8-token", op="i8", T=1, K=1600, N=6400, dtype="f16", gelu=True),
        # a batch of decoding sequences through the down projection of GPT-2 774M
        dict(name="i8-decode-batch", op="i8", T=37, K=5120, N=1280, dtype="bf16", gelu=False),
        # a prompt of odd length through the up projection of GPT-2 355M
        dict(name="i8-prompt", op="i8", T=2047, K=1024, N=4096, dtype="f16", gelu=True),
        # evaluation over a training batch: the down projection of GPT-2 1.5B
        dict(name="i8-batch-1p5b", op="i8", T=32768, K=6400, N=1600, dtype="f16", gelu=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("muon", "orth", "quant", "i8"))
        dtype = rng.choice(("f16", "bf16"))
        if op in ("muon", "orth"):
            case = dict(op=op, count=rng.choice((1, 1, 2, 5, 8)), rows=_log(rng, 48, 6400), cols=_log(rng, 48, 6400),
                        dtype=dtype)
            if op == "muon":
                case.update(nesterov=rng.random() < 0.5, lr=rng.uniform(2e-5, 6e-5))
        elif op == "quant":
            masked = rng.random() < 0.5
            rows, cols = _log(rng, 1, 20000), _log(rng, 16, 6400)
            if masked:
                rows, cols = 4 * (1 + rows // 4), 4 * (cols // 4)
            case = dict(op=op, rows=rows, cols=cols, dtype=dtype, masked=masked)
        else:
            case = dict(op=op, T=_log(rng, 1, 32768), K=16 * _log(rng, 2, 400), N=16 * _log(rng, 2, 400), dtype=dtype,
                        gelu=rng.random() < 0.5)
        if _cost(case) <= most:
            return case


def work(case):
    if case["op"] in ("muon", "orth"):
        m, n = sorted((case["rows"], case["cols"]))
        # per round: the two symmetric products (one triangle each) and the product with X
        flops = case["count"] * STEPS * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n)
        # muon: gradient read, momentum and fp32 weight read and written, 16-bit weight written
        per = 4 + 8 + 8 + 2 if case["op"] == "muon" else 4 + 2
        return {"bytes": case["count"] * m * n * per, "flops": flops}
    if case["op"] == "quant":
        n = case["rows"] * case["cols"]
        return {"bytes": n * 3 + 4 * case["rows"] + (n // 16 if case["masked"] else 0), "flops": 2 * n}
    T, K, N = case["T"], case["K"], case["N"]
    return {"bytes": T * K + N * K + 4 * (T + N) + 2 * T * N, "flops": 2 * T * N * K}


def _gradient(shape, std, gen, dev):
    """A weight gradient's shape of spectrum: columns of unequal size, and a few directions that stand out."""
    count, rows, cols = shape
    g = torch.randn(shape, generator=gen, device=dev)
    g *= torch.exp(0.5 * torch.randn((count, 1, cols), generator=gen, device=dev))
    g += torch.bmm(torch.randn((count, rows, 8), generator=gen, device=dev),
                   torch.randn((count, 8, cols), generator=gen, device=dev)) * (2.0 / math.sqrt(8.0))
    return g * std


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    op = case["op"]
    dtype = DTYPES[case["dtype"]]
    st = dict(case)
    if op in ("muon", "orth"):
        shape = (case["count"], case["rows"], case["cols"])
        st["grad"] = _gradient(shape, 1e-3, gen, dev)
        if op == "muon":
            st["momentum"] = _gradient(shape, 5e-3, gen, dev)
            st["W"] = torch.randn(shape, generator=gen, device=dev) * 0.02
            st["W16"] = st["W"].to(dtype)
            st["scale"] = 0.2 * math.sqrt(max(case["rows"], case["cols"]))   # update of one size for every shape
        else:
            st["out"] = torch.empty(shape, dtype=dtype, device=dev)
        if own:      # the buffer that a program keeps for these calls; the plain form takes none
            import structured_sparse_transformer_b200 as sp
            st["workspace"] = torch.empty(sp.sp24_orthogonalize_size(case["rows"], case["cols"], case["count"]),
                                          dtype=torch.uint8, device=dev)
    elif op == "quant":
        rows, cols = case["rows"], case["cols"]
        x = torch.randn((rows, cols), generator=gen, device=dev)
        x *= torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device=dev))
        st["X"] = x.to(dtype)
        st["q"] = torch.empty((rows, cols), dtype=torch.int8, device=dev)
        st["scale"] = torch.empty(rows, dtype=torch.float32, device=dev)
        st["idx"] = (torch.randint(0, 90, (rows // 4, cols // 4), generator=gen, device=dev).to(torch.uint8)
                     if case["masked"] else None)
    else:
        T, K, N = case["T"], case["K"], case["N"]

        def quantized(rows, std):
            x = torch.randn((rows, K), generator=gen, device=dev) * std
            s = x.abs().amax(1) / 127
            return torch.round(x / s[:, None]).to(torch.int8), s

        st["Xq"], st["sx"] = quantized(T, 1.0)
        st["Wq"], st["sw"] = quantized(N, 0.02)
        st["Y"] = torch.empty((T, N), dtype=dtype, device=dev)
    return st


def _patterns(dev):
    """The 90 4x4 patterns with two ones in every row and column, in the library's order: [90, 4, 4]."""
    pairs = list(itertools.combinations(range(4), 2))
    kept = [p for p in itertools.product(pairs, repeat=4)
            if all(sum(c in row for row in p) == 2 for c in range(4))]
    return torch.tensor([[[c in row for c in range(4)] for row in p] for p in kept], device=dev)


def _dense_mask(idx, rows, cols):
    m = _patterns(idx.device)[idx.long()]                     # [rows/4, cols/4, 4, 4]
    return m.permute(0, 2, 1, 3).reshape(rows, cols)


def _newton_schulz(u):
    norm = u.double().square().sum((1, 2), keepdim=True).sqrt()
    x = (u.double() / (norm + EPS)).float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    for _ in range(STEPS):
        a = x @ x.transpose(1, 2)
        x = A * x + (B * a + C * (a @ a)) @ x
    return x.transpose(1, 2) if tall else x


def _plain(st):
    op = st["op"]
    if op == "orth":
        st["out"].copy_(_newton_schulz(st["grad"]))
        return {"out": st["out"]}
    if op == "muon":
        st["momentum"].mul_(MU).add_(st["grad"])
        u = st["grad"] + MU * st["momentum"] if st["nesterov"] else st["momentum"]
        st["W"].mul_(1.0 - st["lr"] * WEIGHT_DECAY).sub_(_newton_schulz(u) * (st["lr"] * st["scale"]))
        st["W16"].copy_(st["W"])
        return {"momentum": st["momentum"], "W": st["W"], "W16": st["W16"]}
    if op == "quant":
        x = st["X"].float()
        if st["idx"] is not None:
            x = torch.where(_dense_mask(st["idx"], *x.shape), x, torch.zeros_like(x))
        amax = x.abs().amax(1)
        st["scale"].copy_(amax / 127.0)
        inv = torch.where(amax > 0, 127.0 / amax, torch.zeros_like(amax))
        st["q"].copy_(torch.round(x * inv[:, None]))
        return {"q": st["q"], "scale": st["scale"]}
    y = (st["Xq"].float() @ st["Wq"].float().t()) * st["sw"] * st["sx"][:, None]
    if st["gelu"]:
        y = 0.5 * y * torch.erfc(y * -math.sqrt(0.5))
    st["Y"].copy_(y)
    return {"Y": st["Y"]}


def _own(st):
    import structured_sparse_transformer_b200 as sp
    op = st["op"]
    if op == "orth":
        sp.sp24_orthogonalize(st["grad"], st["out"], st["workspace"], steps=STEPS, eps=EPS)
        return {"out": st["out"]}
    if op == "muon":
        sp.sp24_muon_step(st["grad"], st["momentum"], st["W"], st["W16"], st["workspace"], lr=st["lr"], mu=MU,
                          nesterov=st["nesterov"], weight_decay=WEIGHT_DECAY, scale=st["scale"], steps=STEPS, eps=EPS)
        return {"momentum": st["momentum"], "W": st["W"], "W16": st["W16"]}
    if op == "quant":
        sp.sp24_quantize_rows(st["X"], st["q"], st["scale"], st["idx"])
        return {"q": st["q"], "scale": st["scale"]}
    sp.sp24_gemm_i8(st["Xq"], st["sx"], st["Wq"], st["sw"], st["Y"], "gelu" if st["gelu"] else None)
    return {"Y": st["Y"]}


def run(st):
    return _own(st) if own else _plain(st)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op in ("muon", "orth"):
        g = st["grad"].double()
        u = g
        if op == "muon":
            m = MU * st["momentum"].double() + g
            u = g + MU * m if case["nesterov"] else m
        outs = []
        for z in u:                                           # one matrix at a time, on its wide side
            wide = z.shape[0] <= z.shape[1]
            x = z if wide else z.t()
            x = x / (torch.linalg.vector_norm(x) + EPS)
            eye = torch.eye(x.shape[0], dtype=x.dtype, device=x.device)
            for _ in range(STEPS):
                gram = torch.mm(x, x.t())
                x = torch.mm(A * eye + torch.mm(gram, B * eye + C * gram), x)
            outs.append(x if wide else x.t())
        o = torch.stack(outs)
        if op == "orth":
            return {"out": o}
        w = st["W"].double() * (1.0 - case["lr"] * WEIGHT_DECAY) - (case["lr"] * st["scale"]) * o
        return {"momentum": m, "W": w, "W16": w}
    if op == "quant":
        x = st["X"].double()
        if st["idx"] is not None:
            x = x.masked_fill(~_dense_mask(st["idx"], *x.shape), 0.0)
        return {"q": None, "scale": x.abs().max(dim=1).values / 127}
    y = torch.mm(st["Xq"].double(), st["Wq"].double().t())
    y = y * (st["sx"].double()[:, None] * st["sw"].double()[None, :])
    if case["gelu"]:
        y = y * torch.special.ndtr(y)
    return {"Y": y}
