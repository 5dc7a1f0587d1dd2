"""Gated experts (moe_glu_*), CUDA path vs their formulas in 64 bits (GPU).

Two bars per result, both derived from the arithmetic before the first run.

Elementwise: an interval bound carried through the formulas.  u is the largest relative
error of one rounding to the stored type (bf16 2^-8, fp32 2^-24); a sum of K products in
32 bits is off by at most K 2^-23 times the sum of their magnitudes (tensor cores may
truncate, so twice the 2^-24 of a rounding); f and f' are evaluated with an error of at
most 2^-18 max(1, |g|) on top of |f'| <= 1.13 and |f''| <= 0.8 times the error of g.  ReLU's
derivative may fall either way where |g| is within its own error.

Norm: the roundings of independent elements do not add up, so the Frobenius norm of the
error is at most u times the number of roundings on the way (y: h and y; dW2: h and dW2;
dx and dW13: g and u, dg and du, the result, and one for the product of two rounded
factors), relative to the norm of the result; fp32 4 * 2^-24 * sqrt(depth) likewise.
With ReLU, dg of an element whose |g| is within its own error (K 2^-23 sum |x w|, and u |g|)
may be dh u or 0; the two differ by |dh u|, so the norm of those elements' part of dx and of
dW13, sum |dh u| |Wg| and sum |x| |dh u|, is allowed on top.
"""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2, torch.float32: torch.finfo(torch.float32).eps / 2}
ACC = 2.0**-23
EPS_F = 2.0**-18


def make(E, C, M, H, dtype, counts, seed=0, garbage=float("nan")):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda shape, s: torch.empty(shape, dtype=dtype, device="cuda").normal_(0, s, generator=g)  # noqa: E731
    x, dy = rnd((E, C, M), 1.0), rnd((E, C, M), 1.0)
    W13, W2 = rnd((E, M, 2 * H), M**-0.5), rnd((E, H, M), H**-0.5)
    n = torch.tensor(counts, dtype=torch.int32, device="cuda")
    pad = torch.arange(C, device="cuda")[None, :, None] >= n.clamp(0, C)[:, None, None]
    x.masked_fill_(pad, garbage)
    dy.masked_fill_(pad, garbage)
    return x, dy, W13, W2, n


def act(name, g):
    if name == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    if name == "gelu":
        p = torch.special.ndtr(g)
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    return g.clamp(min=0), (g > 0).double()


def reference(x, dy, W13, W2, n, fn):
    """Per expert: the results in 64 bits and elementwise bounds on the kernels' errors."""
    E, C, M = x.shape
    H, u = W2.shape[1], U[x.dtype]
    res = []
    for e in range(E):
        r = max(0, min(int(n[e]), C))
        X, Wg, Wu, W = x[e, :r].double(), W13[e, :, :H].double(), W13[e, :, H:].double(), W2[e].double()
        D = dy[e, :r].double()
        g, v = X @ Wg, X @ Wu
        eg, ev = M * ACC * (X.abs() @ Wg.abs()), M * ACC * (X.abs() @ Wu.abs())
        f, df = act(fn, g)
        efun = EPS_F * g.abs().clamp(min=1)
        h = f * v
        eh = (f.abs() + 1.13 * eg + efun) * (v.abs() + ev) - h.abs()
        eh = eh + u * (h.abs() + eh)
        y = h @ W
        ey = (eh + H * ACC * h.abs()) @ W.abs()
        ey = ey + u * (y.abs() + ey)
        # backward: g and u as stored
        gs, vs = eg + u * (g.abs() + eg), ev + u * (v.abs() + ev)
        dh = D @ W.T
        edh = M * ACC * (D.abs() @ W.abs().T)
        efs = 1.13 * gs + efun
        edf = (g.abs() <= gs).double() if fn == "relu" else 0.8 * gs + efun
        dg, du = dh * v * df, dh * f
        edg = (dh.abs() + edh) * (v.abs() + vs) * (df.abs() + edf) - dg.abs()
        edu = (dh.abs() + edh) * (f.abs() + efs) - du.abs()
        edg, edu = edg + u * (dg.abs() + edg), edu + u * (du.abs() + edu)
        dx = dg @ Wg.T + du @ Wu.T
        edx = (edg + 2 * H * ACC * dg.abs()) @ Wg.abs().T + (edu + 2 * H * ACC * du.abs()) @ Wu.abs().T
        edx = edx + u * (dx.abs() + edx)
        dW13 = torch.cat([X.T @ dg, X.T @ du], 1)
        k = max(r, 1) * ACC
        e13 = torch.cat([X.abs().T @ (edg + k * dg.abs()), X.abs().T @ (edu + k * du.abs())], 1)
        e13 = e13 + u * (dW13.abs() + e13)
        dW2 = h.T @ D
        e2 = (eh + k * h.abs()).T @ D.abs()
        e2 = e2 + u * (dW2.abs() + e2)
        amb = edf * (dh * v).abs() if fn == "relu" else torch.zeros_like(dg)
        s13 = torch.cat([X.abs().T @ amb, torch.zeros_like(X.T @ du)], 1)
        res.append(dict(r=r, y=(y, ey, 0.0), dx=(dx, edx, float((amb @ Wg.abs().T).norm())), dW13=(dW13, e13, float(s13.norm())),
                        dW2=(dW2, e2, 0.0)))
    return res


ROUNDINGS = {"y": 2, "dW2": 2, "dx": 4, "dW13": 4}


def check(name, got, ref, dtype, depth):
    val, err, flips = ref
    d = (got.double() - val).abs()
    tiny = 1e-30
    assert bool(torch.isfinite(got.double()).all()), name
    assert bool((d <= err + tiny).all()), (name, float((d - err).max()))
    if val.numel():
        bar = ROUNDINGS[name] * U[dtype] * (math.sqrt(depth) if dtype == torch.float32 else 1.0)
        assert float(d.norm()) <= bar * float(val.norm()) + flips + tiny, (name, float(d.norm()), float(val.norm()), bar, flips)


CASES = [
    # E, C, M, H, counts
    (1, 1, 64, 64, [1]),
    (1, 1, 64, 64, [0]),
    (2, 3, 64, 128, [3, 0]),
    (3, 37, 128, 192, [37, 1, 20]),
    (4, 65, 192, 64, [64, 65, 63, 0]),
    (1, 333, 320, 448, [333]),
    (5, 130, 256, 320, [129, 128, 127, 130, 2]),
    (2, 257, 64, 576, [256, 257]),
    (3, 600, 512, 256, [511, 0, 513]),
    (3, 40, 64, 64, [-5, 1000, 31]),          # counts outside [0, C] are clamped
    (256, 2, 64, 64, [i % 3 for i in range(256)]),
    (8, 20, 1024, 1088, [0, 1, 20, 17, 0, 16, 3, 2]),
    (32, 1, 512, 1024, [int(i in (9, 13)) for i in range(32)]),
    (3, 100, 576, 704, [100, 64, 1]),
    (2, 128, 192, 1216, [128, 33]),
    (1, 333, 320, 2048, [333]),                                  # few tiles: the depth is cut into shares
    (2, 100, 192, 1216, [100, 33]),
    (1, 3, 64, 2944, [3]),
    (12, 700, 192, 320, [160, 161, 256, 257, 288, 289, 416, 417, 511, 512, 544, 700]),   # last tiles of 1 to 256 rows
    (32, 18, 512, 1024, [(7 * i) % 19 for i in range(32)]),      # long shares: part of the work is fetched
]


def experts(C_max, W13, W2, fn, backward=True):
    from gshard_top_gating_b200.experts import GatedExperts
    ex = GatedExperts(C_max, W13, W2, activation=fn)
    if backward:
        ex.enable_backward()
    return ex


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("fn", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:4])))
def test_forward_and_backward(case, fn, dtype):
    E, C, M, H, counts = case
    x, dy, W13, W2, n = make(E, C, M, H, dtype, counts, seed=E * C + M)
    ex = experts(C, W13, W2, fn)
    mark = 12345.0
    y, dx = torch.full_like(x, mark), torch.full_like(x, mark)
    assert ex(x, n, out=y) is y
    g = ex.backward(x, n, dy, out={"dx": dx})
    ex.check()
    again = ex.backward(x, n, dy)
    ref = reference(x, dy, W13, W2, n, fn)
    for e in range(E):
        r = ref[e]["r"]
        check("y", y[e, :r], ref[e]["y"], dtype, max(M, H))
        check("dx", dx[e, :r], ref[e]["dx"], dtype, max(M, 2 * H))
        check("dW13", g["dW13"][e], ref[e]["dW13"], dtype, max(M, r))
        check("dW2", g["dW2"][e], ref[e]["dW2"], dtype, max(M, r))
        assert bool((y[e, r:] == mark).all()) and bool((dx[e, r:] == mark).all()), "rows past the last one"
        assert torch.equal(again["dx"][e, :r], dx[e, :r])
    assert torch.equal(again["dW13"], g["dW13"]) and torch.equal(again["dW2"], g["dW2"])
    ex.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_inference_equals_training_forward(dtype):
    x, dy, W13, W2, n = make(4, 300, 128, 384, dtype, [300, 17, 0, 256])
    a, b = experts(300, W13, W2, "silu", backward=False), experts(512, W13, W2, "silu")
    ya, yb = torch.zeros_like(x), torch.zeros_like(x)
    assert torch.equal(a(x, n, out=ya), b(x, n, out=yb))
    x, n = x[:, :40].contiguous(), n.clamp(max=39)
    ya, yb = torch.zeros_like(x), torch.zeros_like(x)
    assert torch.equal(a(x, n, out=ya), b(x, n, out=yb))


def test_shorter_batches_than_the_handle_holds_and_no_rows_at_all():
    x, dy, W13, W2, n = make(3, 200, 128, 128, torch.bfloat16, [200, 3, 90])
    ex = experts(200, W13, W2, "silu")
    for C in (200, 91, 4):
        xs = x[:, :C].contiguous()
        y = torch.zeros_like(xs)
        ex(xs, n, out=y)          # counts above C are clamped
        ref = reference(xs, dy[:, :C], W13, W2, n, "silu")
        for e in range(3):
            check("y", y[e, :ref[e]["r"]], ref[e]["y"], torch.bfloat16, 128)
            assert not y[e, ref[e]["r"]:].any()
    x0 = x[:, :0].contiguous()
    assert ex(x0, n).shape == (3, 0, 128)
    g = ex.backward(x0, n, x0)
    assert not g["dW13"].any() and not g["dW2"].any()


def test_experts_without_rows_are_skipped_on_request():
    x, dy, W13, W2, n = make(4, 70, 64, 192, torch.bfloat16, [70, 0, 5, 0])
    ex = experts(70, W13, W2, "gelu")
    ex(x, n)
    dense = ex.backward(x, n, dy)
    mark = {"dW13": torch.full_like(W13, 7.0), "dW2": torch.full_like(W2, 7.0)}
    ex.backward(x, n, dy, out=mark, skip_empty_experts=True)
    for k in ("dW13", "dW2"):
        for e in range(4):
            want = dense[k][e] if int(n[e]) else torch.full_like(dense[k][e], 7.0)
            assert torch.equal(mark[k][e], want)
            assert int(n[e]) or not dense[k][e].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_captured_step_replays_on_new_data(dtype):
    E, C, M, H = 3, 150, 128, 320
    x, dy, W13, W2, n = make(E, C, M, H, dtype, [150, 0, 66])
    x2, dy2, _, _, n2 = make(E, C, M, H, dtype, [31, 150, 64], seed=9)
    ex = experts(C, W13, W2, "silu")
    y = torch.zeros_like(x)
    out = {"dx": torch.zeros_like(x), "dW13": torch.empty_like(W13), "dW2": torch.empty_like(W2)}
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ex(x, n, out=y)
        ex.backward(x, n, dy, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ex(x, n, out=y)
        ex.backward(x, n, dy, out=out)
    x.copy_(x2)
    dy.copy_(dy2)
    n.copy_(n2)
    graph.replay()
    torch.cuda.synchronize()
    ref = experts(C, W13, W2, "silu")
    y_ref = ref(x2, n2)
    g_ref = ref.backward(x2, n2, dy2)
    for e in range(E):
        r = int(n2[e])
        assert torch.equal(y[e, :r], y_ref[e, :r]) and torch.equal(out["dx"][e, :r], g_ref["dx"][e, :r])
    assert torch.equal(out["dW13"], g_ref["dW13"]) and torch.equal(out["dW2"], g_ref["dW2"])


def test_two_handles_on_two_streams():
    a = make(2, 140, 128, 256, torch.bfloat16, [140, 70], seed=1)
    b = make(2, 140, 128, 256, torch.bfloat16, [9, 133], seed=2)
    exs = [experts(140, t[2], t[3], "silu") for t in (a, b)]
    want = [(ex(t[0], t[4], out=torch.zeros_like(t[0])), ex.backward(t[0], t[4], t[1])) for ex, t in zip(exs, (a, b))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [(ex(t[0], t[4], out=torch.zeros_like(t[0]), stream=s), ex.backward(t[0], t[4], t[1], stream=s))
               for ex, t, s in zip(exs, (a, b), streams)]
        torch.cuda.synchronize()
        for (y, g), (yw, gw), t in zip(got, want, (a, b)):
            assert torch.equal(y, yw) and torch.equal(g["dW13"], gw["dW13"]) and torch.equal(g["dW2"], gw["dW2"])
            for e in range(2):
                assert torch.equal(g["dx"][e, :int(t[4][e])], gw["dx"][e, :int(t[4][e])])


@pytest.mark.parametrize("fn", ["silu", "gelu"])
def test_gradients_against_differences(fn):
    """<dy, y(W + t d)> differentiated numerically (fp32, central differences) against the
    gradients along d.  Truncation t^2 |third derivative| / 6 and the rounding of y over 2t
    are both below 1e-3 of the derivative at t = 2^-7."""
    E, C, M, H = 2, 33, 64, 128
    x, dy, W13, W2, n = make(E, C, M, H, torch.float32, [33, 12], garbage=0.0)
    ex = experts(C, W13, W2, fn)
    ex(x, n)
    g = ex.backward(x, n, dy)
    live = torch.arange(C, device="cuda")[None, :, None] < n[:, None, None]
    gen = torch.Generator(device="cuda").manual_seed(3)

    def loss(x, W13, W2):
        e2 = experts(C, W13, W2, fn, backward=False)
        y = e2(x, n, out=torch.zeros_like(x))
        return float((y.double() * dy.double() * live).sum())

    t = 2.0**-7
    for name, ten in (("dx", x), ("dW13", W13), ("dW2", W2)):
        # a direction along the gradient's signs, scaled to the tensor, has a large derivative
        d = torch.sign(torch.where(live, g["dx"], torch.zeros_like(x)) if name == "dx" else g[name]) * ten.abs().mean()
        d = d * torch.rand(d.shape, generator=gen, device="cuda")
        up, dn = ten + t * d, ten - t * d
        args = lambda v: tuple(v if k == name else o for k, o in (("dx", x), ("dW13", W13), ("dW2", W2)))  # noqa: E731
        num = (loss(*args(up)) - loss(*args(dn))) / (2 * t)
        grad = torch.where(live, g["dx"], torch.zeros_like(x)) if name == "dx" else g[name]
        ana = float((grad.double() * d.double()).sum())
        assert abs(num - ana) <= 1e-2 * abs(ana), (name, num, ana)


def test_refusals():
    from gshard_top_gating_b200 import _lib as L
    from gshard_top_gating_b200.experts import GatedExperts
    x, dy, W13, W2, n = make(2, 40, 64, 128, torch.bfloat16, [40, 3])
    ex = GatedExperts(40, W13, W2)
    with pytest.raises(L.MoeError) as err:
        ex.backward(x, n, dy)                      # before enable_backward
    assert err.value.status == L.MOE_ERR_STATE
    ex(x, n)
    ex.enable_backward()
    with pytest.raises(L.MoeError) as err:
        ex.backward(x, n, dy)                      # that forward kept nothing
    assert err.value.status == L.MOE_ERR_STATE
    ex(x, n)
    ex.backward(x, n, dy)
    with pytest.raises(L.MoeError) as err:
        ex.backward(x[:, :39].contiguous(), n, dy[:, :39].contiguous())
    assert err.value.status == L.MOE_ERR_STATE
    with pytest.raises(L.MoeError) as err:
        ex(torch.zeros(2, 41, 64, dtype=torch.bfloat16, device="cuda"), n)
    assert err.value.status == L.MOE_ERR_INVALID_ARG
    for bad in (x.float(), x[:, :, :32].contiguous(), x.transpose(0, 1), x[:1].contiguous(), x.cpu(), x[0]):
        with pytest.raises(ValueError):
            ex(bad, n)
    for bad in (n.long(), n[:1], n.cpu()):
        with pytest.raises(ValueError):
            ex(x, bad)
    with pytest.raises(ValueError):
        ex(x, n, out=torch.empty_like(x[:, :20]))
    with pytest.raises(ValueError):
        GatedExperts(40, W13, W2, activation="tanh")
    with pytest.raises(ValueError):
        GatedExperts(40, W13, W2[:, :64].contiguous())
    with pytest.raises(TypeError):
        GatedExperts(40, W13.half(), W2.half())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("C", [5, 300])
def test_nan_and_infinity_in_a_row_stay_in_that_row(C, dtype):
    x, dy, W13, W2, n = make(2, C, 128, 192, dtype, [C, C - 1])
    ex = experts(C, W13, W2, "silu")
    clean, g_clean = ex(x, n, out=torch.zeros_like(x)), ex.backward(x, n, dy, out={"dx": torch.zeros_like(x)})
    x[0, 3, 7], x[1, 2, 0], dy[1, 1, 5] = float("nan"), float("inf"), float("nan")
    y, g = ex(x, n, out=torch.zeros_like(x)), ex.backward(x, n, dy, out={"dx": torch.zeros_like(x)})
    hit_y, hit_dx = {(0, 3), (1, 2)}, {(0, 3), (1, 2), (1, 1)}
    for e in range(2):
        for r in range(int(n[e])):
            assert ((e, r) in hit_y) == bool(y[e, r].isnan().any()), (e, r)
            assert ((e, r) in hit_dx) == bool(g["dx"][e, r].isnan().any()), (e, r)
            if (e, r) not in hit_y:
                assert torch.equal(y[e, r], clean[e, r])
            if (e, r) not in hit_dx:
                assert torch.equal(g["dx"][e, r], g_clean["dx"][e, r])


def test_saturated_gates():
    """|g| from 20 to 1e4: f(g) is g or (nearly) 0, never NaN, for every f."""
    E, C, M, H = 1, 4, 64, 64
    W13 = torch.zeros(E, M, 2 * H, dtype=torch.bfloat16, device="cuda")
    W13[0, :, :H] = torch.eye(M, H)
    W13[0, :, H:] = torch.eye(M, H)
    W2 = torch.eye(H, M, dtype=torch.bfloat16, device="cuda")[None].contiguous()
    x = torch.tensor([20.0, 90.0, 128.0, 1e4], device="cuda").bfloat16()[None, :, None].repeat(1, 1, M).contiguous()
    n = torch.tensor([4], dtype=torch.int32, device="cuda")
    for fn in ("silu", "gelu", "relu"):
        for sign in (1.0, -1.0):
            ex = experts(C, W13, W2, fn)
            y = ex(sign * x, n)
            g = ex.backward(sign * x, n, torch.ones_like(x))
            want = x.double() ** 2 if sign > 0 else torch.zeros_like(x.double())
            assert bool(((y.double() - want).abs() <= 2.0**-7 * want + 1e-5).all()), (fn, sign)
            assert g["dx"].isfinite().all() and g["dW13"].isfinite().all()


@pytest.mark.parametrize("fn", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("C", [8, 70], ids=["few rows", "tiles"])
def test_gradients_of_rows_of_any_magnitude(C, fn):
    """g and u between the passes hold 16 bits: fp16 for 32 columns that fit it, else bf16,
    the first of 32 then with a rounding of 2u.  Rows of magnitudes from 1e-9 to 1e9, a row of
    zeros, and one whose u are past fp16's range in one column in 32 only: dx of each row
    within the bar of `check` and 1/32 of a rounding more, dW13 of all of them (twice the
    interval bound, since that first one's error is twice the u it counts)."""
    M, H = 64, 192
    x, dy, W13, W2, n = make(1, C, M, H, torch.bfloat16, [C], seed=C)
    scales = torch.tensor([1.0, 1e-9, 1e9, 1e-5, 3e5, 0.0, 1.0, 300.0], device="cuda").repeat(C // 8 + 1)[:C]
    x = (x.float() * scales[None, :, None]).bfloat16()
    W13[0, :, H + 5::32] *= 2.0**14
    ex = experts(C, W13, W2, fn)
    ex(x, n)
    g = ex.backward(x, n, dy)
    ref = reference(x, dy, W13, W2, n, fn)[0]
    u = U[torch.bfloat16]
    bar = (ROUNDINGS["dx"] + 1 / 32) * u
    val, err, _ = ref["dx"]
    for i in range(C):
        slack = float(err[i].norm()) if fn == "relu" else 0.0       # either side of 0 (see check's flips)
        assert float((g["dx"][0, i].double() - val[i]).norm()) <= bar * float(val[i].norm()) + slack + 1e-30, (i, float(scales[i]))
    assert bool(((g["dW13"][0].double() - ref["dW13"][0]).abs() <= 2 * ref["dW13"][1] + 1e-30).all())


def test_offsets_past_32_bits():
    """x and y of more than 2^31 elements: rows at the far end of both experts."""
    E, C, M, H = 2, 1_060_000, 1024, 64
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB")
    assert E * C * M > 2**31
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(E, C, M, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    W13 = torch.empty(E, M, 2 * H, dtype=torch.bfloat16, device="cuda").normal_(0, M**-0.5, generator=g)
    W2 = torch.empty(E, H, M, dtype=torch.bfloat16, device="cuda").normal_(0, H**-0.5, generator=g)
    n = torch.tensor([C, C - 77], dtype=torch.int32, device="cuda")
    y = experts(C, W13, W2, "silu", backward=False)(x, n, out=torch.full_like(x, 7.0))
    for e, rows in ((0, [0, 1, C // 2, C - 1]), (1, [0, C // 2, C - 79, C - 78])):
        gu = x[e, rows].double() @ W13[e].double()
        want = (act("silu", gu[:, :H])[0] * gu[:, H:]) @ W2[e].double()
        got = y[e, rows].double()
        assert float((got - want).norm() / want.norm()) <= 2 * U[torch.bfloat16]
    assert bool((y[1, C - 77:] == 7.0).all())


def test_misaligned_pointers_are_refused():
    from gshard_top_gating_b200 import _lib as L
    x, dy, W13, W2, n = make(1, 8, 64, 64, torch.bfloat16, [8])
    ex = experts(8, W13, W2, "silu")
    buf = torch.zeros(x.numel() + 8, dtype=torch.bfloat16, device="cuda")
    off = buf[1:1 + x.numel()].view(1, 8, 64)
    for args, kw in (((off, n), {}), ((x, n), {"out": off})):
        with pytest.raises(L.MoeError) as err:
            ex(*args, **kw)
        assert err.value.status == L.MOE_ERR_INVALID_ARG
    ex(x, n)
    with pytest.raises(L.MoeError) as err:
        ex.backward(x, n, off)
    assert err.value.status == L.MOE_ERR_INVALID_ARG
