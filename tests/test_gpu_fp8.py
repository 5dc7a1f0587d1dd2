"""8-bit products with a scale for each block of 128 (moe_fp8_*), CUDA path vs formulas (GPU).

The quantiser's values are compared bit for bit with the same three roundings made on the
CPU in fp32 (448 / a, its product with x, e4m3 to nearest even); the scales are within half
a step of a / 448.

The product: K exact products of 8-bit values times their scales, added in 32 bits (at most
K 2^-23 of the sum of their magnitudes; tensor cores may truncate), two roundings for the
scales, one rounding to bf16 (2^-8 of the value).  In norm the single rounding is all that
remains: 1.05 * 2^-8.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

U = torch.finfo(torch.bfloat16).eps / 2
TINY = 2.0**-100


def cpu_blocks(x):
    R, K = x.shape
    nb = (K + 127) // 128
    return torch.nn.functional.pad(x.float(), (0, nb * 128 - K)).view(R, nb, 128)


def cpu_quantize(x):
    """x [R, K] on the CPU -> (q as e4m3, amax of each block)."""
    R, K = x.shape
    f = cpu_blocks(x)
    a = f.abs().amax(2).clamp(min=TINY)
    q = (f * (torch.full_like(a, 448.0) / a)[:, :, None]).reshape(R, -1)[:, :K]
    return q.to(torch.float8_e4m3fn), a


def bits(q):
    return q.cpu().contiguous().view(torch.uint8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 16), (1, 128), (3, 144), (7, 112), (61, 1456), (130, 7168), (1000, 256)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_quantize_rows(shape, dtype):
    from gshard_top_gating_b200.fp8 import quantize_rows
    g = torch.Generator().manual_seed(shape[0] + shape[1])
    x = torch.randn(shape, generator=g) * torch.exp(3 * torch.randn(shape[0], 1, generator=g))
    x[:, ::61] *= 30
    x[0, : shape[1] // 2] = 0.0                      # zeros, whole blocks of them in wide rows
    x[-1] *= 1e-35                                   # below the floor of the scale
    x = x.to(dtype)
    q, s = quantize_rows(x.cuda())
    qr, a = cpu_quantize(x)
    assert torch.equal(bits(q), bits(qr))
    want = a.double() / 448
    assert bool(((s.cpu().double() - want).abs() <= 2.0**-24 * want).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_quantize_rows_of_infinities_and_nans(dtype):
    from gshard_top_gating_b200.fp8 import quantize_rows
    x = torch.ones(4, 272, dtype=dtype)
    x[0, 5] = float("nan")
    x[1, 130] = float("inf")
    x[2, 271] = float("-inf")
    x[3, 0], x[3, 1] = torch.finfo(dtype).max, torch.finfo(dtype).min
    q, s = quantize_rows(x.cuda())
    q, s = q.cpu().float(), s.cpu()
    assert q[0, :128].isnan().all() and s[0, 0].isnan() and not q[0, 128:].isnan().any()
    assert s[1, 1].isinf() and q[1, 130].isnan() and (q[1, 131:256] == 0).all() and s[1, 0] == torch.tensor(1.0) / 448
    assert s[2, 2].isinf() and q[2, 271].isnan() and not q[2, :256].isnan().any()
    assert q[3, 0] == 448 and q[3, 1] == -448 and s[3, 0].isfinite()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 16, 8), (2, 128, 128), (3, 144, 264), (1, 1456, 2008), (2, 64, 40)],
                         ids=lambda s: "x".join(map(str, s)))
def test_quantize_weights(shape, dtype):
    from gshard_top_gating_b200.fp8 import quantize_weights
    E, K, N = shape
    g = torch.Generator().manual_seed(K + N)
    W = (torch.randn(shape, generator=g) * K**-0.5).to(dtype)
    W[0, : min(K, 128), : min(N, 128)] = 0
    q, s = quantize_weights(W.cuda())
    assert q.shape == (E, N, K) and s.shape == (E, (N + 127) // 128, (K + 127) // 128)
    f = W.float().transpose(1, 2)
    for i in range(s.shape[1]):
        for j in range(s.shape[2]):
            blk = f[:, 128 * i:128 * (i + 1), 128 * j:128 * (j + 1)]
            a = blk.abs().amax((1, 2)).clamp(min=TINY)
            want = (blk * (torch.full_like(a, 448.0) / a)[:, None, None]).to(torch.float8_e4m3fn)
            assert torch.equal(bits(q[:, 128 * i:128 * (i + 1), 128 * j:128 * (j + 1)]), bits(want))
            assert bool(((s[:, i, j].cpu().double() - a.double() / 448).abs() <= 2.0**-24 * a.double() / 448).all())


def values(q, s, rows):
    """The numbers that q and s stand for, in 64 bits; s has a scale for each `rows` x 128 block."""
    K = q.shape[-1]
    s = s.double().repeat_interleave(128, -1)[..., :K]
    if rows > 1:
        s = s.repeat_interleave(rows, -2)[..., : q.shape[-2], :]
    return q.double() * s


def make(E, C, K, N, counts, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    def e4m3(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    def scale(*shape):
        return torch.exp(torch.randn(shape, generator=g, device="cuda"))
    nk, nn = (K + 127) // 128, (N + 127) // 128
    n = torch.tensor(counts, dtype=torch.int32, device="cuda")
    pad = torch.arange(C, device="cuda")[None, :, None] >= n.clamp(0, C)[:, None, None]
    xq, xs = e4m3(E, C, K), scale(E, C, nk)
    # rows that nobody wrote: NaN bytes and NaN scales
    xq = torch.where(pad, torch.full_like(xq.view(torch.uint8), 0x7F), xq.view(torch.uint8)).view(torch.float8_e4m3fn)
    return xq, xs.masked_fill(pad, float("nan")), e4m3(E, N, K), scale(E, nn, nk) * K**-0.5, n


CASES = [
    # E, C, K, N, counts
    (1, 1, 16, 8, [1]),
    (1, 1, 128, 128, [0]),
    (2, 5, 144, 264, [5, 0]),
    (3, 33, 256, 120, [33, 1, 20]),
    (1, 333, 1456, 2008, [333]),
    (4, 130, 384, 512, [129, 128, 127, 2]),
    (2, 300, 2048, 136, [257, 300]),
    (3, 40, 112, 72, [-5, 1000, 31]),        # counts outside [0, C] are clamped
    (256, 2, 128, 16, [i % 3 for i in range(256)]),
    (3, 600, 7168, 256, [511, 0, 600]),
    (4, 17, 7168, 520, [17, 0, 1, 16]),
    (16, 64, 2048, 384, [64, 33, 0, 1] * 4),
    (1, 1, 4096, 1024, [1]),
    (2, 30, 1168, 264, [30, 19]),
    (1, 333, 4112, 520, [333]),                              # few tiles: the depth is cut into shares
    (2, 130, 3088, 1000, [129, 7]),
    (1, 100, 4096, 512, [100]),
    (1, 300, 656, 4088, [300]),                              # tiles of 128 columns
    (3, 200, 384, 3208, [200, 0, 161]),
    (6, 300, 272, 1640, [300, 32, 257, 64, 0, 96]),          # of 256
    (1, 160, 7168, 200, [160]),                              # of 64, in shares
    (5, 260, 528, 328, [256, 260, 32, 96, 40]),              # of 64, more than one block of 256 rows
    (32, 9, 2048, 1544, [i % 10 for i in range(32)]),        # long shares: part of the work is fetched
]


def product(C, wq, ws):
    from gshard_top_gating_b200.fp8 import Fp8Matmul
    return Fp8Matmul(C, wq, ws)


def check_product(y, xq, xs, wq, ws, n, K):
    for e in range(xq.shape[0]):
        r = max(0, min(int(n[e]), xq.shape[1]))
        X, W = values(xq[e, :r], xs[e, :r], 1), values(wq[e], ws[e], 128)
        want, mag = X @ W.T, X.abs() @ W.abs().T
        err = (K * 2.0**-23 + 2.0**-22) * mag
        err = err + U * (want.abs() + err)
        d = (y[e, :r].double() - want).abs()
        assert bool((d <= err).all()), (e, float((d / err.clamp(min=1e-300)).max()))
        if r:
            rel = float(d.norm() / want.norm())
            assert rel <= 1.05 * U, (e, rel)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:4])))
def test_product(case):
    E, C, K, N, counts = case
    xq, xs, wq, ws, n = make(*case, seed=K + N)
    mm = product(C, wq, ws)
    y = torch.full((E, C, N), 12345.0, dtype=torch.bfloat16, device="cuda")
    assert mm(xq, xs, n, out=y) is y
    mm.check()
    check_product(y, xq, xs, wq, ws, n, K)
    for e in range(E):
        assert bool((y[e, max(0, min(counts[e], C)):] == 12345.0).all()), "rows past the last one"
    y2 = torch.full_like(y, 12345.0)
    assert torch.equal(mm(xq, xs, n, out=y2), y)


def test_shorter_batches_than_the_handle_holds_and_no_rows_at_all():
    xq, xs, wq, ws, n = make(3, 200, 272, 328, [200, 3, 90])
    mm = product(200, wq, ws)
    for C in (200, 91, 4):
        a, b = xq[:, :C].contiguous(), xs[:, :C].contiguous()
        y = torch.zeros(3, C, 328, dtype=torch.bfloat16, device="cuda")
        mm(a, b, n, out=y)
        check_product(y, a, b, wq, ws, n, 272)
    assert mm(xq[:, :0].contiguous(), xs[:, :0].contiguous(), n).shape == (3, 0, 328)


def test_one_expert_of_infinite_scale_and_nan_stays_apart():
    """NaN and infinite scales of one expert's rows and weights reach that expert's rows only."""
    xq, xs, wq, ws, n = make(3, 50, 256, 256, [50, 50, 50])
    xs[1, 7, 0], ws[1, 1, 1] = float("nan"), float("inf")
    y = product(50, wq, ws)(xq, xs, n)
    assert y[1, 7].isnan().all() and not y[1, :7, :128].isnan().any()
    assert not y[1, :7, 128:].isfinite().any()
    for e in (0, 2):
        assert y[e].isfinite().all()


def test_quantize_and_multiply_together():
    """bf16 rows and weights through both quantisers and the product, against the bf16
    product in 64 bits.  A value of a block with largest a is off by at most half a step of
    e4m3, 2^-4 of itself, or of its smallest normal, 2^-10 a / 448; so a product of two by
    2 (2^-4) + 2^-8 of its magnitude and that floor: in norm 2^-4 sqrt(2) / sqrt(3) at most
    over the roundings' uniform spread, 0.0511, plus bf16's."""
    from gshard_top_gating_b200.fp8 import quantize_rows, quantize_weights
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(2, 150, 640, generator=g, device="cuda").bfloat16()
    W = (torch.randn(2, 640, 384, generator=g, device="cuda") * 640**-0.5).bfloat16()
    n = torch.tensor([150, 77], dtype=torch.int32, device="cuda")
    xq, xs = quantize_rows(x)
    y = product(150, *quantize_weights(W))(xq, xs, n)
    for e in range(2):
        r = int(n[e])
        want = x[e, :r].double() @ W[e].double()
        assert float((y[e, :r].double() - want).norm() / want.norm()) <= 0.0511 + U


def test_captured_replay_streams_and_two_handles():
    xq, xs, wq, ws, n = make(2, 100, 256, 384, [100, 30])
    xq2, xs2, wq2, ws2, n2 = make(2, 100, 256, 384, [5, 99], seed=8)
    mm, mm2 = product(100, wq, ws), product(100, wq2, ws2)
    new = lambda: torch.zeros(2, 100, 384, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    want, want2 = mm(xq, xs, n, out=new()), mm2(xq2, xs2, n2, out=new())
    y = new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mm(xq, xs, n, out=y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    xq.view(torch.uint8).copy_(xq2.view(torch.uint8))
    xs.copy_(xs2)
    n.copy_(n2)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, mm(xq2, xs2, n2, out=new()))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        o1, o2 = new(), new()
        torch.cuda.synchronize()
        mm(xq2, xs2, n2, out=o1, stream=a)
        mm2(xq2, xs2, n2, out=o2, stream=b)
        torch.cuda.synchronize()
        assert torch.equal(o1, y) and torch.equal(o2, want2)


def test_refusals():
    from gshard_top_gating_b200 import _lib as L
    from gshard_top_gating_b200.fp8 import Fp8Matmul, quantize_rows, quantize_weights
    xq, xs, wq, ws, n = make(2, 40, 256, 128, [40, 3])
    mm = Fp8Matmul(40, wq, ws)
    for a, b, c in ((xq.float(), xs, n), (xq[:1].contiguous(), xs, n), (xq, xs[:, :, :1].contiguous(), n), (xq, xs, n.long()),
                    (xq.cpu(), xs, n), (xq, xs.double(), n), (xq[0], xs, n)):
        with pytest.raises(ValueError):
            mm(a, b, c)
    with pytest.raises(ValueError):
        mm(xq, xs, n, out=torch.empty(2, 40, 128, device="cuda"))
    bigger = make(2, 41, 256, 128, [1, 1])
    with pytest.raises(L.MoeError) as err:
        mm(bigger[0], bigger[1], bigger[4])
    assert err.value.status == L.MOE_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        Fp8Matmul(40, wq, ws[:, :, :1].contiguous())
    with pytest.raises(L.MoeError):
        quantize_rows(torch.zeros(3, 24, device="cuda"))          # K not a multiple of 16
    with pytest.raises(L.MoeError):
        quantize_weights(torch.zeros(1, 32, 12, device="cuda"))   # N not a multiple of 8
    with pytest.raises(TypeError):
        quantize_rows(torch.zeros(3, 32, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        quantize_rows(torch.zeros(32, 3, device="cuda").t())
    q, s = quantize_rows(torch.zeros(0, 32, device="cuda"))
    assert q.shape == (0, 32) and s.shape == (0, 1)


def test_offsets_past_32_bits():
    """Rows of more than 2^31 values through the quantiser and the product."""
    from gshard_top_gating_b200.fp8 import quantize_rows, quantize_weights
    R, K, N = 300_100, 7168, 64
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB")
    assert R * K > 2**31
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(R, K, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    q, s = quantize_rows(x)
    rows = [0, 1, R // 2, R - 2, R - 1]
    qr, a = cpu_quantize(x[rows].cpu())
    assert torch.equal(bits(q[rows]), bits(qr))
    W = torch.empty(1, K, N, dtype=torch.bfloat16, device="cuda").normal_(0, K**-0.5, generator=g)
    wq, ws = quantize_weights(W)
    n = torch.tensor([R - 1], dtype=torch.int32, device="cuda")
    y = product(R, wq, ws)(q[None], s[None], n, out=torch.full((1, R, N), 7.0, dtype=torch.bfloat16, device="cuda"))
    for r in rows[:-1]:
        want = values(q[r:r + 1], s[r:r + 1], 1) @ values(wq[0], ws[0], 128).T
        assert float((y[0, r].double() - want[0]).norm() / want.norm()) <= 1.05 * U
    assert bool((y[0, R - 1] == 7.0).all())


def test_misaligned_pointers_are_refused():
    from gshard_top_gating_b200 import _lib as L
    from gshard_top_gating_b200.fp8 import quantize_rows
    buf = torch.zeros(64 * 4 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(L.MoeError) as err:
        quantize_rows(buf[1:257].view(4, 64))
    assert err.value.status == L.MOE_ERR_INVALID_ARG
    xq, xs, wq, ws, n = make(1, 4, 64, 64, [4])
    raw = torch.zeros(4 * 64 + 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(L.MoeError) as err:
        product(4, wq, ws)(raw[1:257].view(torch.float8_e4m3fn).view(1, 4, 64), xs, n)
    assert err.value.status == L.MOE_ERR_INVALID_ARG
