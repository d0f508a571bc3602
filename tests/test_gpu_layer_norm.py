"""GPU tests of the layer norm, its gradient and the norm into the block-scaled layer, against oracle/fp8.py (fp64).

Bounds, derived from the formulas (u = 2^-24, half an fp32 step; sums of a row run over at most 16 values a lane, 6 lane
steps and 16 waves, fewer than 40 additions deep, so a sum's error is at most 40 u of the sum of the magnitudes):
* mean: the first mean is corrected by the sum of the differences to it, so that what stays is one rounding of the mean
  and of each x - p: u |mean| + 42 u mean|x - mean|, and the latter is at most 42 u / rstd;
* rstd: the mean of squares within 44 u, square root, quotient, eps: 50 u of rstd;
* z = (x - mean) rstd: rstd times the mean's error, and 54 u |z|;
* y = z w + beta: |w| times z's error, 2 u |z w|, u |y|; bf16: half a step, 2^-8 of the value;
* dx, from the same mean and rstd: g one rounding (two with 1 + gamma), z two, the two sums 46 u of the mean magnitudes:
  rstd u (6 |g| + 50 mean|g| + 54 |z| mean|g z|);
* dgamma, dbeta: no more additions in a row than n, the rows: u (n + 6) sum |terms|.
"""
import numpy as np
import pytest

from gpu_helpers import log

from bit_diffusion_model_amd import svdq
from oracle import fp8 as o
from test_gpu_fp8 import check, codes, dev, dtype, weights
from test_gpu_int8 import at_any_value, host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _torch():
    import torch

    return torch


def make(B, S, C, dt, seed, pad=0, mean=0.0):
    """Rows of normals, each of its own magnitude, with outlier channels, about `mean`."""
    torch = _torch()
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((B, S, C)) * 10.0 ** rng.uniform(-2, 2, (B, S, 1))
    x[..., rng.choice(C, max(1, C // 50), replace=False)] *= 30.0
    t = torch.from_numpy((x + mean).astype(np.float32)).to("cuda:0").to(dtype(dt))
    buf = torch.full((B, S, C + pad), float("nan"), dtype=t.dtype, device="cuda:0")
    buf[..., :C] = t
    return buf[..., :C]


def params(B, C, each, seed):
    rng = np.random.default_rng(seed)
    shape = (B, C) if each else (C,)
    return (1 + 0.3 * rng.standard_normal(shape)).astype(np.float32), rng.standard_normal(shape).astype(np.float32)


def wide(t, each):
    return None if t is None else t[:, None, :].astype(np.float64) if each else t.astype(np.float64)


def check_norm(Y, X, g, b, each, eps, one, stats=None, what=""):
    x, gw, bw = host(X), wide(g, each), wide(b, each)
    y, mean, rstd = o.layer_norm(x, gw, bw, eps, one)
    z = (x - mean[..., None]) * rstd[..., None]
    w = o._weight(gw, one)
    em = U * np.abs(mean) + 42 * U / rstd
    ez = rstd[..., None] * em[..., None] + 54 * U * np.abs(z)
    tol = np.abs(w) * ez + 2 * U * np.abs(z * w) + 2 * U * (np.abs(y) + np.abs(z * w)) + 1e-37
    if Y.dtype == _torch().bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(y)
    err = np.abs(host(Y) - y) / tol
    assert (err <= 1).all(), f"{what}: worst {err.max()} of the bound"
    if stats is not None:
        m, r = (host(t).reshape(mean.shape) for t in stats)
        assert (np.abs(m - mean) <= em + 1e-37).all() and (np.abs(r - rstd) <= 50 * U * rstd).all(), what
    return err.max()


SHAPES = [(1, 1, 1), (1, 3, 2), (2, 5, 7), (1, 77, 16), (3, 41, 100), (2, 9, 128), (1, 50, 129), (2, 33, 200), (1, 7, 256),
          (2, 30, 264), (3, 5, 511), (1, 19, 512), (2, 11, 520), (1, 300, 1024), (2, 7, 1111), (1, 6, 2048), (2, 40, 2944),
          (1, 5, 4097), (1, 3, 8192), (2, 2, 12300), (1, 2, 16384), (1, 5000, 96), (1, 3000, 640), (7, 1, 1280)]


@pytest.mark.parametrize("B,S,C", SHAPES)
@pytest.mark.parametrize("dt,yd", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("each", [False, True])
def test_norm(B, S, C, dt, yd, each):
    torch = _torch()
    X = make(B, S, C, dt, B + S + C, pad=(0, 8, 3)[S % 3])
    g, b = params(B, C, each, C)
    ln = svdq.LayerNorm(C, g, b, 1e-5, one_plus=each)
    stats = ln.alloc_stats(X)
    Y = ln.forward(X, {"bf16": svdq.BF16, "f32": svdq.F32}[yd], stats=stats)
    check_norm(Y, X, g, b, each, 1e-5, each, stats, f"{B}x{S}x{C}")
    assert torch.equal(ln.forward(X, {"bf16": svdq.BF16, "f32": svdq.F32}[yd]), Y)


@pytest.mark.parametrize("C", [24, 300, 1280, 5000])
def test_norm_far_means(C):
    """A mean far from zero costs its own rounding only; constant rows give beta to the bit, whatever the value."""
    torch = _torch()
    X = make(1, 9, C, "f32", C, mean=3e4)
    g, b = params(1, C, False, C)
    ln = svdq.LayerNorm(C, g, b, 1e-5)
    check_norm(ln.forward(X, svdq.F32), X, g, b, False, 1e-5, False, None, "far mean")
    rows = torch.tensor([3000.7, -1e-3, 0.0, 7.1e5, 1 / 3], device="cuda:0").view(1, 5, 1).expand(1, 5, C).contiguous()
    Y = ln.forward(rows, svdq.F32)
    assert torch.equal(Y, ln.beta.expand(1, 5, C))


@pytest.mark.parametrize("C", [40, 700, 3000])
def test_norm_nan_rows_and_no_weights(C):
    """A row with a NaN or an infinity is lost, its neighbours are not; gamma and beta may be missing."""
    torch = _torch()
    X = make(2, 12, C, "f32", C)
    X[0, 3, C // 2] = float("nan")
    X[1, 7, C - 1] = float("inf")
    clean = X.clone()
    clean[0, 3], clean[1, 7] = 1.0, 1.0
    for g, b in ((None, None), (params(2, C, False, 1)[0], None), (None, params(2, C, True, 1)[1])):
        ln = svdq.LayerNorm(C, g, b, one_plus=g is None)
        Y, Z = ln.forward(X, svdq.F32), ln.forward(clean, svdq.F32)
        assert Y[0, 3].isnan().all() and Y[1, 7].isnan().all()
        Y[0, 3], Y[1, 7], Z[0, 3], Z[1, 7] = 0, 0, 0, 0
        assert torch.equal(Y, Z)
        q, s = ln.quantize(X)
        assert s[:, 3].isnan().all() and s[:, 19].isnan().all() and (codes(q)[[3, 19]] == 0).all()
        assert torch.isfinite(s[:, [0, 1, 2, 4, 18, 20]]).all()


@pytest.mark.parametrize("B,S,C", [(2, 5, 7), (3, 41, 100), (2, 30, 264), (2, 7, 1111), (2, 3, 5001)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strides_and_places(B, S, C, dt):
    """Rows at any value, images interleaved or one and the same, in place: the bits of the contiguous call, and nothing
    written beside the rows."""
    torch = _torch()
    X = make(B, S, C, dt, C).contiguous()
    g, b = params(B, C, True, C)
    ln = svdq.LayerNorm(C, g, b)
    yd = svdq.F32 if dt == "f32" else svdq.BF16
    stats = ln.alloc_stats(X)
    Y = ln.forward(X, yd, stats=stats)
    dY = make(B, S, C, dt, C + 1).contiguous()
    want = ln.backward(dY, X, stats)
    for strides in ((S * (C + 1) + 3, C + 1, 1), (C, B * C, 1)):
        _, x = at_any_value((B, S, C), strides, X.dtype, float("nan"))
        x.copy_(X)
        buf, y = at_any_value((B, S, C), strides, X.dtype, 7.0)
        ln.forward(x, yd, out=y)
        assert torch.equal(y, Y)
        _, d = at_any_value((B, S, C), strides, X.dtype, float("nan"))
        d.copy_(dY)
        got = ln.backward(d, x, stats, out=y)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
        y.fill_(7.0)
        assert (buf == 7.0).all(), "a value beside the rows was written"
        assert torch.equal(ln.backward(d, x, stats, out=d)[0], want[0])
        d.copy_(dY)
        x2 = x.clone()
        ln.forward(x, yd, out=x)
        assert torch.equal(x, Y)
        assert torch.equal(ln.backward(d, x2, stats, out=x2)[0], want[0])
    same = X[:1].expand(B, S, C)
    assert torch.equal(ln.forward(same, yd), ln.forward(same.contiguous(), yd))


@pytest.mark.parametrize("B,S,C", SHAPES)
@pytest.mark.parametrize("dt,dd", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("each", [False, True])
def test_gradient(B, S, C, dt, dd, each):
    torch = _torch()
    X, dY = make(B, S, C, dt, B + S + C, pad=(0, 8, 3)[S % 3]), make(B, S, C, dd, S * C, pad=(3, 0, 8)[S % 3])
    g, b = params(B, C, each, C)
    ln = svdq.LayerNorm(C, g, b, 1e-5, one_plus=each)
    stats = ln.alloc_stats(X)
    ln.forward(X, stats=stats)
    dX, dg, db = ln.backward(dY, X, stats)
    x, dy = host(X), host(dY)
    mean, rstd = (host(t).reshape(B, S) for t in stats)
    dx, dyz, _ = o.layer_norm_grad(dy, x, mean, rstd, wide(g, each), each)
    r = rstd[..., None]
    z, gg = (x - mean[..., None]) * r, dy * o._weight(wide(g, each), each)
    tol = r * U * (6 * np.abs(gg) + 50 * np.abs(gg).mean(-1, keepdims=True)
                   + 54 * np.abs(z) * np.abs(gg * z).mean(-1, keepdims=True)) + 3 * U * np.abs(dx) + 1e-37
    if dt == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(dx)
    err = np.abs(host(dX) - dx) / tol
    assert (err <= 1).all(), f"dX: worst {err.max()} of the bound"
    over, n = (1 if each else (0, 1)), (S if each else B * S)
    assert tuple(dg.shape) == tuple(db.shape) == g.shape
    for got, terms in ((dg, dyz), (db, dy)):
        err = np.abs(host(got) - terms.sum(over)) / (U * (n + 6) * np.abs(terms).sum(over) + 1e-37)
        assert (err <= 1).all(), f"column sums: worst {err.max()} of the bound"
    again = ln.backward(dY, X, stats)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dg) and torch.equal(again[2], db)
    only = ln.backward(dY, X, stats, weights=False)
    assert torch.equal(only[0], dX) and only[1] is None and only[2] is None


@pytest.mark.parametrize("B,S,C,each", [(1, 20000, 64, False), (3, 20001, 200, True), (2, 9000, 1500, False), (1, 70001, 16, False)])
def test_gradient_many_rows(B, S, C, each):
    """Many blocks to a run: the column sums against sums in 64 bits on the device."""
    torch = _torch()
    X, dY = make(B, S, C, "bf16", 1), make(B, S, C, "f32", 2)
    g, b = params(B, C, each, C)
    ln = svdq.LayerNorm(C, g, b)
    stats = ln.alloc_stats(X)
    ln.forward(X, stats=stats)
    _, dg, db = ln.backward(dY, X, stats)
    z = (X.double() - stats[0].double().view(B, S, 1)) * stats[1].double().view(B, S, 1)
    over, n = (1 if each else (0, 1)), (S if each else B * S)
    for got, t in ((dg, dY.double() * z), (db, dY.double())):
        bound = U * (n + 6) * t.abs().sum(over) + 1e-37
        assert ((got.double() - t.sum(over)).abs() <= bound).all()


@pytest.mark.parametrize("C", [12, 300, 1200])
def test_gradient_against_differences(C):
    """The gradient along a random direction against the difference of two forward passes in fp32."""
    torch = _torch()
    gen = torch.Generator(device="cuda:0").manual_seed(C)
    x, v, u = (torch.randn(1, 6, C, device="cuda:0", generator=gen) for _ in range(3))
    g, b = params(1, C, False, C)
    ln = svdq.LayerNorm(C, g, b, 1e-3)
    stats = ln.alloc_stats(x)
    ln.forward(x, svdq.F32, stats=stats)
    dx, _, _ = ln.backward(v, x, stats)
    h = 2.0 ** -6  # truncation about h^2, rounding about 2^-24 / h: both below 1e-3 of the values
    diff = ((ln.forward(x + h * u, svdq.F32).double() - ln.forward(x - h * u, svdq.F32).double()) * v.double()).sum(2) / (2 * h)
    got = (dx.double() * u.double()).sum(2)
    scale = (dx.double().norm(dim=2) * u.double().norm(dim=2))
    assert ((diff - got).abs() <= 2e-3 * scale).all()


def test_no_rows():
    torch = _torch()
    for shape, each in (((0, 64), False), ((2, 0, 64), True), ((2, 0, 64), False), ((0, 5, 64), False)):
        B = shape[0] if len(shape) == 3 else 1
        g, b = params(B, 64, each, 0)
        ln = svdq.LayerNorm(64, g, b)
        X = torch.empty(shape, device="cuda:0")
        stats = ln.alloc_stats(X)
        assert ln.forward(X, stats=stats).shape == X.shape
        dX, dg, db = ln.backward(X, X, stats)
        assert dX.shape == X.shape and (dg == 0).all() and (db == 0).all() and tuple(dg.shape) == g.shape
        q, s = ln.quantize(X)
        assert q.shape == (0, 128)


def test_checked():
    torch = _torch()
    g, b = params(2, 64, True, 0)
    ln, X = svdq.LayerNorm(64, g, b), torch.ones(2, 5, 64, device="cuda:0")
    st = ln.alloc_stats(X)
    bad = [lambda: ln.forward(X[:1]), lambda: ln.forward(X[..., :60]), lambda: ln.forward(X.half()), lambda: ln.forward(X.cpu()),
           lambda: ln.forward(X, svdq.BF16_GELU), lambda: ln.forward(X, out=torch.empty(2, 5, 64, device="cuda:0")),
           lambda: ln.forward(X, stats=(st[0][:5], st[1])), lambda: ln.forward(X, stats=(st[0].double(), st[1])),
           lambda: ln.backward(X[:1], X, st), lambda: ln.backward(X, X, None), lambda: ln.backward(X, X, (st[0].cpu(), st[1])),
           lambda: ln.backward(X, X, st, out=torch.empty(2, 5, 64, device="cuda:0", dtype=torch.bfloat16)),
           lambda: ln.forward(X, svdq.F32, out=X[:1].expand(2, 5, 64)),
           lambda: svdq.LayerNorm(64, g, b[:1]), lambda: svdq.LayerNorm(60, g, b), lambda: svdq.LayerNorm(0),
           lambda: svdq.LayerNorm(64, eps=0.0).forward(X)]
    for i, f in enumerate(bad):
        with pytest.raises(svdq.SvdqError):
            f()
            log(f"call {i} was taken")
            if i == 15:
                svdq.LayerNorm(0).forward(X[..., :0])


@pytest.mark.parametrize("B,S,C,N", [(1, 3, 100, 50), (2, 77, 768, 300), (1, 40, 2944, 130), (3, 100, 130, 257), (2, 9, 9000, 64)])
@pytest.mark.parametrize("dt,yd", [("bf16", "f32"), ("f32", "gelu")])
def test_norm_and_layer(B, S, C, N, dt, yd):
    """The norm's codes against the oracle's norm in fp64 (a value beside a border may take the code on its other side), and
    the layer on them bit for bit the two calls."""
    torch = _torch()
    X = make(B, S, C, dt, C, pad=3)
    g, b = params(B, C, True, N)
    ln = svdq.LayerNorm(C, g, b, one_plus=True)
    qW, sW, bias = weights(N, C, N)
    lin = svdq.Fp8Linear(qW, sW, C, bias=bias)
    ydtype = {"f32": svdq.F32, "gelu": svdq.BF16_GELU}[yd]
    stats = ln.alloc_stats(X)
    q, s = ln.quantize(X, stats=stats)
    st2 = ln.alloc_stats(X)
    Y = ln.forward_linear(X, lin, ydtype, stats=st2)
    assert torch.equal(Y, lin.gemm(q, s, ydtype)) and torch.equal(st2[0], stats[0]) and torch.equal(st2[1], stats[1])
    check(Y, codes(q), s.cpu().numpy(), qW, sW, bias, ydtype, "norm and layer")
    # codes of the kernel's own fp32 output are the quantizer's, bit for bit
    y32 = ln.forward(X, svdq.F32)
    q2, s2 = svdq.quantize_act_fp8(y32.view(B * S, C))
    M = B * S
    assert torch.equal(s2[:, :M], s[:, :M]) and np.array_equal(codes(q2), codes(q))
    check_norm(y32, X, g, b, True, 1e-5, True, stats, "norm before codes")


def test_block_forward_and_backward():
    """The run of them as a user would: norm into the layer, the gradient of the layer's input, the norm's gradient; on a
    captured graph too, replayed between eager calls."""
    torch = _torch()
    B, S, C, N = 2, 50, 300, 500
    rng = np.random.default_rng(0)
    g, b = params(B, C, True, 0)
    ln = svdq.LayerNorm(C, g, b, one_plus=True)
    lin = svdq.Fp8Linear(*o.pack_weights(rng.standard_normal((C, N)) / np.sqrt(C)), C)
    back = lin.transposed()
    xs = [make(B, S, C, "bf16", i).contiguous() for i in range(3)]
    dys = [torch.from_numpy(rng.standard_normal((B * S, N)).astype(np.float32)).cuda() for _ in range(3)]

    def step(x, dy):
        stats = ln.alloc_stats(x)
        y = ln.forward_linear(x, lin, svdq.BF16, stats=stats)
        dz = back.forward(dy, svdq.F32)
        return (y, dz, *ln.backward(dz.view(B, S, C), x, stats))

    want = [step(x, dy) for x, dy in zip(xs, dys)]
    # against fp32 torch on the layer's own weights: the codes' rounding is what differs, 2^-4 of a value at most
    w = torch.from_numpy(o.values(*o.pack_weights(np.random.default_rng(0).standard_normal((C, N)) / np.sqrt(C)), 128)[:, :C]).float().cuda()
    x = xs[0].float().requires_grad_()
    gt, bt = (torch.from_numpy(t).cuda()[:, None].requires_grad_() for t in (g, b))
    y = (torch.nn.functional.layer_norm(x, (C,)) * (1 + gt) + bt).view(-1, C) @ w.t()
    y.backward(dys[0])
    for name, got, ref in (("y", want[0][0], y), ("dx", want[0][2], x.grad), ("dgamma", want[0][3], gt.grad[:, 0]),
                           ("dbeta", want[0][4], bt.grad[:, 0])):
        off = float((got.float() - ref.detach()).norm() / ref.detach().norm())
        log(f"block: {name} off by {off:.2e}")
        assert off <= 2.0 ** -4
    x, dy = xs[0].clone(), dys[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, dy)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        dy.copy_(dys[i])
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(out, want[i]):
            assert torch.equal(got, ref)
        step(xs[2], dys[2])
        torch.cuda.synchronize()


def test_example_runs_and_its_gradients():
    """examples/modulated_block_fp8.py: norm, two layers and back through them; the codes' error of y and each gradient."""
    import importlib.util
    import os
    import sys
    from unittest import mock

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "modulated_block_fp8.py")
    spec = importlib.util.spec_from_file_location("modulated_block_fp8", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    with mock.patch.object(sys, "argv", ["x", "--images", "2", "--rows", "77", "--channels", "320"]):
        errors = m.main()
    # a code is off by at most 2^-4 of its value, 2^-4 / sqrt(3) in the mean square; a product has two such operands, and y
    # and each gradient come through two products and a GELU or its derivative at a value that is off by one product's error
    assert sorted(errors) == ["dscale", "dshift", "dx", "y"]
    assert max(errors.values()) < 3 * np.sqrt(2) * 2.0 ** -4 / np.sqrt(3)
