"""The operators that the framework's benchmark of operators measures, case by case, with their plain forms.

Three operators of an expert layer, on rows that are already sorted into per-expert
buffers [E, C, width] with a count of rows for each expert (rows past it are memory that
nobody wrote):

  glu_forward   y = (f(x Wg) * (x Wu)) W2            gated experts, W13 = [Wg | Wu]
  glu_step      the same forward and its backward    dx, dW13, dW2 for an upstream dy
  fp8_matmul    y = (xq * xs) (wq * ws)^T            e4m3 values, a scale for each 1 x 128 block
                                                     of x and each 128 x 128 block of w
  fp8_quantize  q, s of the rows of x                a scale for each 1 x 128 block

`run` computes them in plain torch operations, or, with `own` set, by the framework's
entry points.
"""
import math

import torch

own = False

#: Largest value of e4m3, and the amax below which a block is scaled as if it had this one.
E4M3_MAX, TINY = 448.0, 2.0**-100
BLOCK = 128


def listed():
    return [
        # one token of a 32-expert layer: two experts hold one row each, the others none
        dict(name="glu one token", op="glu_forward", dtype="bf16", act="silu", E=32, C=1, M=1024, H=4096, active=2, fill=0.25),
        # a decode batch of 64 tokens with two choices each over the same experts
        dict(name="glu decode batch", op="glu_forward", dtype="bf16", act="silu", E=32, C=13, M=1024, H=4096, active=31, fill=0.25),
        # the mid layer's batch: capacity factor 2, about half of the slots taken, odd counts
        dict(name="glu mid", op="glu_forward", dtype="bf16", act="gelu", E=32, C=1024, M=1024, H=4096, active=32, fill=0.1),
        # the large layer's experts on one of four GPUs, at capacity
        dict(name="glu large", op="glu_forward", dtype="bf16", act="silu", E=16, C=2048, M=2048, H=8192, active=16, fill=0.9),
        # the tiny layer in 32 bits: parity work, where launches count
        dict(name="glu step tiny f32", op="glu_step", dtype="f32", act="silu", E=8, C=80, M=64, H=256, active=8, fill=0.4),
        # a training step of a few of the mid layer's experts, one of them empty, an odd capacity
        dict(name="glu step mid", op="glu_step", dtype="bf16", act="silu", E=8, C=683, M=1024, H=4096, active=7, fill=0.25),
        # a training step of the large layer's experts on one of eight GPUs
        dict(name="glu step large", op="glu_step", dtype="bf16", act="gelu", E=8, C=2048, M=2048, H=8192, active=8, fill=0.9),
        # the wide layer's first product for a decode batch, 32 of 256 experts on this GPU
        dict(name="fp8 decode batch", op="fp8_matmul", E=32, C=8, K=7168, N=4096, active=28, fill=0.25),
        # a dense projection whose last blocks are cut short
        dict(name="fp8 odd", op="fp8_matmul", E=1, C=333, K=1456, N=2008, active=1, fill=1.0),
        # the wide layer's first product for a prefill batch, a part of this GPU's experts
        dict(name="fp8 prefill", op="fp8_matmul", E=16, C=2048, K=7168, N=4096, active=16, fill=0.9),
        # the rows of a decode batch
        dict(name="fp8 quantize few", op="fp8_quantize", dtype="bf16", R=61, K=7168),
        # the rows of the wide layer's batch
        dict(name="fp8 quantize batch", op="fp8_quantize", dtype="bf16", R=65536, K=7168),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glu_forward", "glu_forward", "glu_step", "fp8_matmul", "fp8_matmul", "fp8_quantize"])
    if op == "fp8_quantize":
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), R=_log(rng, 1, 32768), K=16 * _log(rng, 1, 448))
    E = _log(rng, 1, 32)
    active = max(1, min(E, rng.randint(1, E) if rng.random() < 0.5 else E))
    C, fill = _log(rng, 1, 2048), round(rng.uniform(0.0, 1.0), 2)
    while True:
        if op == "fp8_matmul":
            K, N = 16 * _log(rng, 1, 448), 8 * _log(rng, 1, 896)
            if E * K * N <= 2**29 and E * C * (K + N) <= 2**28 and 2.0 * E * C * K * N <= 1.2e12:
                return dict(op=op, E=E, C=C, K=K, N=N, active=active, fill=fill)
            continue
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        M, H = 64 * _log(rng, 1, 32), 64 * _log(rng, 1, 128)
        most = 1.2e12 if dtype == "bf16" else 2e10
        if 6.0 * E * C * M * H * (3 if op == "glu_step" else 1) <= most and E * M * H <= 2**28:
            return dict(op=op, dtype=dtype, act=rng.choice(["silu", "gelu"]), E=E, C=C, M=M, H=H, active=active, fill=fill)
        C, E = max(1, C // 2), max(1, E // 2)
        active = min(active, E)


# ------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32


def _counts(case):
    """Rows of each expert: `active` of them hold some, from `fill` of the capacity up, spread over the experts; of
    three or more one is full and one holds a single row."""
    E, C, a = case["E"], case["C"], case["active"]
    g = torch.Generator().manual_seed(E * 1000003 + C)
    n = torch.zeros(E, dtype=torch.int64)
    which = torch.randperm(E, generator=g)[:a]
    lo = max(1, int(case["fill"] * C))
    n[which] = torch.randint(lo, C + 1, (a,), generator=g)
    if a >= 3:
        n[which[0]], n[which[1]] = C, 1
    return n.to(torch.int32)


def _normal(g, shape, scale, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)


def _quantize(x):
    """Rows of x in e4m3 with a scale for each block of 128 columns."""
    R, K = x.shape
    nb = (K + BLOCK - 1) // BLOCK
    f = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - K)).view(R, nb, BLOCK)
    amax = f.abs().amax(dim=2).clamp(min=TINY)
    q = (f * (E4M3_MAX / amax)[:, :, None]).view(R, nb * BLOCK)[:, :K].to(torch.float8_e4m3fn)
    return q, amax / E4M3_MAX


def _quantize_tiles(w):
    """w [E, N, K] in e4m3 with a scale for each 128 x 128 block."""
    E, N, K = w.shape
    q, s = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device=w.device), []
    for e in range(E):
        nn, nk = (N + BLOCK - 1) // BLOCK, (K + BLOCK - 1) // BLOCK
        f = torch.nn.functional.pad(w[e].float(), (0, nk * BLOCK - K, 0, nn * BLOCK - N)).view(nn, BLOCK, nk, BLOCK)
        amax = f.abs().amax(dim=(1, 3)).clamp(min=TINY)
        f = f * (E4M3_MAX / amax)[:, None, :, None]
        q[e] = f.reshape(nn * BLOCK, nk * BLOCK)[:N, :K].to(torch.float8_e4m3fn)
        s.append(amax / E4M3_MAX)
    return q, torch.stack(s)


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "fp8_quantize":
        x = _normal(g, (case["R"], case["K"]), 1.0, _dtype(case))
        x[:, :: 61] *= 20.0      # the few wide channels that activations have
        return {"x": x}
    E, C = case["E"], case["C"]
    n = _counts(case).cuda()
    pad = torch.arange(C, device="cuda")[None, :, None] >= n[:, None, None]
    if case["op"] == "fp8_matmul":
        K, N = case["K"], case["N"]
        x = _normal(g, (E * C, K), 1.0, torch.bfloat16)
        x[:, :: 61] *= 20.0
        xq, xs = _quantize(x)
        wq, ws = _quantize_tiles(_normal(g, (E, N, K), K**-0.5, torch.bfloat16))
        xq, xs = xq.view(E, C, K), xs.view(E, C, -1).masked_fill(pad, float("nan"))
        return {"n": n, "pad": pad, "xq": xq, "xs": xs, "wq": wq, "ws": ws}
    M, H, dt = case["M"], case["H"], _dtype(case)
    s = {"n": n, "pad": pad, "act": case["act"], "H": H}
    s["x"] = _normal(g, (E, C, M), 1.0, dt).masked_fill_(pad, float("nan"))
    s["W13"] = _normal(g, (E, M, 2 * H), M**-0.5, dt)
    s["W2"] = _normal(g, (E, H, M), H**-0.5, dt)
    if case["op"] == "glu_step":
        s["dy"] = _normal(g, (E, C, M), 1.0, dt).masked_fill_(pad, float("nan"))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op = s["op"] = case["op"]
    if op == "fp8_quantize":
        R, K = s["x"].shape
        s["q"] = torch.empty(R, K, dtype=torch.float8_e4m3fn, device="cuda")
        s["s"] = torch.empty(R, (K + BLOCK - 1) // BLOCK, device="cuda")
    elif op == "fp8_matmul":
        s["y"] = torch.zeros(case["E"], case["C"], case["N"], dtype=torch.bfloat16, device="cuda")
    else:
        s["y"] = torch.zeros_like(s["x"])
        if op == "glu_step":
            s["grads"] = {"dx": torch.zeros_like(s["x"]), "dW13": torch.empty_like(s["W13"]), "dW2": torch.empty_like(s["W2"])}
    if own:
        if op == "fp8_matmul":
            from gshard_top_gating_b200.fp8 import Fp8Matmul
            s["plan"] = Fp8Matmul(case["C"], s["wq"], s["ws"])
        elif op != "fp8_quantize":
            from gshard_top_gating_b200.experts import GatedExperts
            s["plan"] = GatedExperts(case["C"], s["W13"], s["W2"], activation=case["act"])
            if op == "glu_step":
                s["plan"].enable_backward()
    return s


# ------------------------------------------------------------------ one pass

def _act(name, g):
    """f(g) and f'(g)."""
    if name == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    c = 0.5 * (1.0 + torch.erf(g * 0.5**0.5))
    return g * c, c + g * torch.exp(-0.5 * g * g) * (2.0 * math.pi) ** -0.5


def _glu(s):
    H, dt = s["H"], s["x"].dtype
    x = s["x"].float().masked_fill(s["pad"], 0.0)
    W13, W2 = s["W13"].float(), s["W2"].float()
    gu = torch.bmm(x, W13)
    g, u = gu[:, :, :H], gu[:, :, H:]
    f, df = _act(s["act"], g)
    h = f * u
    y = torch.bmm(h, W2).to(dt)
    if s["op"] == "glu_forward":
        return {"y": y}
    dy = s["dy"].float().masked_fill(s["pad"], 0.0)
    dh = torch.bmm(dy, W2.transpose(1, 2))
    dgu = torch.cat([dh * u * df, dh * f], dim=2)
    return {"y": y, "dx": torch.bmm(dgu, W13.transpose(1, 2)).to(dt), "dW13": torch.bmm(x.transpose(1, 2), dgu).to(dt),
            "dW2": torch.bmm(h.transpose(1, 2), dy).to(dt)}


def _fp8_matmul(s):
    xs = s["xs"].masked_fill(s["pad"], 0.0)
    E, C, K = s["xq"].shape
    N = s["wq"].shape[1]
    x = s["xq"].float() * xs.repeat_interleave(BLOCK, dim=2)[:, :, :K]
    w = s["wq"].float() * s["ws"].repeat_interleave(BLOCK, dim=1)[:, :N].repeat_interleave(BLOCK, dim=2)[:, :, :K]
    return {"y": torch.bmm(x, w.transpose(1, 2)).to(torch.bfloat16)}


def run(s):
    op = s["op"]
    if own:
        if op == "fp8_quantize":
            from gshard_top_gating_b200.fp8 import quantize_rows
            quantize_rows(s["x"], out=(s["q"], s["s"]))
            return {"q": s["q"], "s": s["s"]}
        if op == "fp8_matmul":
            return {"y": s["plan"](s["xq"], s["xs"], s["n"], out=s["y"])}
        y = s["plan"](s["x"], s["n"], out=s["y"])
        if op == "glu_forward":
            return {"y": y}
        g = s["plan"].backward(s["x"], s["n"], s["dy"], out=s["grads"])
        return {"y": y, "dx": g["dx"], "dW13": g["dW13"], "dW2": g["dW2"]}
    if op == "fp8_quantize":
        q, sc = _quantize(s["x"])
        return {"q": q, "s": sc}
    return _fp8_matmul(s) if op == "fp8_matmul" else _glu(s)


def work(case):
    if case["op"] == "fp8_quantize":
        R, K, es = case["R"], case["K"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": R * (K * (es + 1) + 4 * ((K + 127) // 128)), "flops": 2 * R * K}
    n = _counts(case)
    rows, busy = int(n.sum()), int((n > 0).sum())
    if case["op"] == "fp8_matmul":
        K, N = case["K"], case["N"]
        nk, nn = (K + 127) // 128, (N + 127) // 128
        return {"bytes": busy * (K * N + 4 * nk * nn) + rows * (K + 4 * nk + 2 * N), "flops": 2 * rows * K * N}
    M, H, es = case["M"], case["H"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "glu_forward":
        return {"bytes": es * (3 * busy * M * H + 2 * rows * M), "flops": 6 * rows * M * H}
    # weights once, x and dy in, y and dx out, every weight's gradient out (zeros for an idle expert)
    return {"bytes": es * (3 * (busy + case["E"]) * M * H + 4 * rows * M), "flops": 18 * rows * M * H}


# ------------------------------------------------------------------ the same in 64 bits, expert by expert

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "fp8_quantize":
        x = s["x"].double()
        sc = torch.stack([b.abs().max(dim=1).values.clamp(min=TINY) for b in x.split(BLOCK, dim=1)], dim=1) / E4M3_MAX
        return {"q": None, "s": sc}
    n = s["n"].tolist()
    E, C = case["E"], case["C"]
    if case["op"] == "fp8_matmul":
        K, N = case["K"], case["N"]
        y = torch.zeros(E, C, N, dtype=torch.float64, device="cuda")
        for e, r in enumerate(n):
            for k0 in range(0, K, BLOCK):
                k1 = min(K, k0 + BLOCK)
                p = s["xq"][e, :r, k0:k1].double() @ s["wq"][e, :, k0:k1].double().T
                ws = s["ws"][e, :, k0 // BLOCK].double()[torch.arange(N, device="cuda") // BLOCK]
                y[e, :r] += p * s["xs"][e, :r, k0 // BLOCK].double()[:, None] * ws[None, :]
        return {"y": y}
    M, H = case["M"], case["H"]
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out = {"y": zeros(E, C, M)}
    if case["op"] == "glu_step":
        out |= {"dx": zeros(E, C, M), "dW13": zeros(E, M, 2 * H), "dW2": zeros(E, H, M)}
    for e, r in enumerate(n):
        x, Wg, Wu, W2 = s["x"][e, :r].double(), s["W13"][e, :, :H].double(), s["W13"][e, :, H:].double(), s["W2"][e].double()
        g, u = x @ Wg, x @ Wu
        if case["act"] == "silu":
            p = torch.sigmoid(g)
            df = p + g * p * (1 - p)
        else:
            p = torch.special.ndtr(g)
            df = p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        h = g * p * u
        out["y"][e, :r] = h @ W2
        if case["op"] == "glu_step":
            dy = s["dy"][e, :r].double()
            dh = dy @ W2.T
            dg, du = dh * u * df, dh * g * p
            out["dx"][e, :r] = dg @ Wg.T + du @ Wu.T
            out["dW13"][e, :, :H], out["dW13"][e, :, H:], out["dW2"][e] = x.T @ dg, x.T @ du, h.T @ dy
    return out
