"""GPU layer normalisation and its gradients against the formulas in 64 bits
and, for the gradients, against differences of the 64-bit forward pass.

Tolerances (relative L2 per output), fixed before the first run: a result
that is rounded once to a type of p significand bits is off by at most 2^-p;
the fp32 arithmetic before it adds a few roundings of 2^-24 per element plus
a sum's tree of log2(dim) roundings: 64 * 2^-24 covers both.  dw and db are
sums over rows of terms of either sign, compared against the norm of what
they sum (sqrt(rows) times a term), hence the same bound.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f64": torch.float64, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0 ** -24, "f64": 2.0 ** -53, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
EPS = 1e-5


def tol(kind, acc="f32"):
    return HALF_ULP[kind] + 64 * (2.0 ** -53 if acc == "f64" else 2.0 ** -24)


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


def rand(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape))


def rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    n = b.norm()
    return float((a - b).norm() / n) if n > 0 else float((a - b).norm())


def forward64(x, w, b, eps=EPS):
    mu = x.mean(-1, keepdim=True)
    var = ((x - mu) ** 2).mean(-1, keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    y = (x - mu) * r
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y, mu[..., 0], r[..., 0]


def backward64(dy, x, w, mu, r):
    xh = (x - mu[:, None]) * r[:, None]
    d = dy if w is None else dy * w
    dx = r[:, None] * (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


SHAPES = [(1, 1), (3, 2), (1, 7), (5, 31), (9, 32), (2, 255), (700, 256), (33, 257), (4, 500),
          (7, 513), (3, 1000), (1300, 1024), (2, 1025), (5, 2048), (5, 2047), (3, 4096), (3, 4100),
          (2, 8192), (2, 8191), (2, 8193), (3, 20000), (1, 33333)]


@pytest.mark.parametrize("kind,wkind", [("f32", "f32"), ("f64", "f64"), ("bf16", "bf16"),
                                        ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_forward_and_backward(fg, rows, dim, kind, wkind):
    x = (rand(1, rows, dim) * 2 + 3 * rand(2, rows, 1)).to(TYPES[kind])
    w = (1 + 0.2 * rand(3, dim)).to(TYPES[wkind])
    b = rand(4, dim).to(TYPES[wkind])
    dy = rand(5, rows, dim).to(TYPES[kind])
    xc, wc, bc, dyc = (t.cuda() for t in (x, w, b, dy))
    y, mean, rstd = fg.layer_norm(xc, wc, bc, EPS)
    y64, mu64, r64 = forward64(x.double(), w.double(), b.double())
    assert y.dtype == x.dtype and y.shape == x.shape
    assert rel(mean, mu64) <= tol("f32", kind)
    # rstd amplifies the variance's error by half of var / (var + eps)
    assert rel(rstd, r64) <= tol("f64" if kind == "f64" else "f32", kind)
    assert rel(y, y64) <= tol(kind, kind)
    dx, dw, db = fg.layer_norm_backward(dyc, xc, wc, mean, rstd)
    # against the formula on the statistics that the forward pass returned
    dx64, dw64, db64 = backward64(dy.double(), x.double(), w.double(), mean.double().cpu(),
                                  rstd.double().cpu())
    size = (dy.double().norm() * rstd.double().cpu().max())
    assert float((dx.double().cpu() - dx64).norm()) <= tol(kind, kind) * float(
        max(dx64.norm(), size)) + 1e-300
    xh = (x.double() - mean.double().cpu()[:, None]) * rstd.double().cpu()[:, None]
    for got, want, terms in ((dw, dw64, dy.double() * xh), (db, db64, dy.double())):
        assert got.dtype == w.dtype
        assert float((got.double().cpu() - want).norm()) <= tol(wkind, kind) * float(
            max(want.norm(), terms.norm())) + 1e-300


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_without_weight_or_bias(fg, weight, bias):
    x, dy = rand(1, 37, 200).float(), rand(2, 37, 200).float()
    w = rand(3, 200).float() if weight else None
    b = rand(4, 200).float() if bias else None
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    y, mean, rstd = fg.layer_norm(x.cuda(), cu(w), cu(b))
    d = lambda t: None if t is None else t.double()  # noqa: E731
    y64, mu64, r64 = forward64(x.double(), d(w), d(b))
    assert rel(y, y64) <= tol("f32")
    dx, dw, db = fg.layer_norm_backward(dy.cuda(), x.cuda(), cu(w), mean, rstd, bias=bias)
    dx64, dw64, db64 = backward64(dy.double(), x.double(), d(w), mu64, r64)
    assert rel(dx, dx64) <= tol("f32")
    assert (dw is None) == (not weight) and (db is None) == (not bias)
    if weight:
        assert rel(dw, dw64) <= tol("f32")
    if bias:
        assert rel(db, db64) <= tol("f32")


def test_gradient_against_differences(fg):
    # d/dt of sum(dy * y) along a random direction, central differences of
    # the 64-bit forward pass: step h leaves h^2 ~ 1e-8 of curvature.
    x, dy, w, b = rand(1, 6, 40), rand(2, 6, 40), 1 + 0.2 * rand(3, 40), rand(4, 40)
    y, mean, rstd = fg.layer_norm(x.cuda(), w.cuda(), b.cuda())
    dx, dw, db = fg.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    h = 1e-5
    for i, grad in ((0, dx), (1, dw), (2, db)):
        args = [x, w, b]
        way = rand(9 + i, *args[i].shape)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * way, args[i] - h * way
        slope = ((forward64(*up)[0] - forward64(*down)[0]) * dy).sum() / (2 * h)
        assert abs(float(slope) - float((grad.cpu() * way).sum())) <= 1e-7 * (1 + abs(float(slope)))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim,ld,skip", [(64, 80, 0), (64, 67, 3), (3001, 3008, 1), (2048, 2064, 8)])
def test_strided_and_unaligned_rows(fg, kind, dim, ld, skip):
    big = rand(1, 20, ld + skip).to(TYPES[kind]).cuda()
    x = big[:, skip:skip + dim]
    dyb = rand(2, 20, ld + skip).to(TYPES[kind]).cuda()
    dy = dyb[:, :dim]
    w = (1 + 0.1 * rand(3, dim)).float().cuda()
    keep = big.clone()
    y, mean, rstd = fg.layer_norm(x, w, w)
    y64, mu64, r64 = forward64(x.double().cpu(), w.double().cpu(), w.double().cpu())
    assert rel(y, y64) <= tol(kind)
    dx, dw, db = fg.layer_norm_backward(dy, x, w, mean, rstd)
    dx64, dw64, db64 = backward64(dy.double().cpu(), x.double().cpu(), w.double().cpu(), mu64, r64)
    assert rel(dx, dx64) <= tol(kind) and rel(dw, dw64) <= tol("f32") and rel(db, db64) <= tol("f32")
    assert torch.equal(big, keep)


def test_in_place_and_higher_axes(fg):
    x = rand(1, 3, 5, 96).float().cuda()
    y, mean, rstd = fg.layer_norm(x)
    assert mean.shape == (3, 5) and y.shape == x.shape
    z = x.clone()
    fg.layer_norm(z, out=z)
    assert torch.equal(z, y)
    # permuted axes: rows at no single stride are copied
    p = x.permute(1, 0, 2)
    assert torch.equal(fg.layer_norm(p)[0], y.permute(1, 0, 2))


def test_a_large_level_costs_no_digits_of_the_variance(fg):
    # mean 1000, deviation 1: E[x^2] - mean^2 in fp32 would leave 1e6 * 2^-24
    # = 6% of the variance in doubt; about the mean only x's own rounding
    # (2^-24 * 1000 absolute) counts.
    x = (1000 + rand(1, 4, 4096)).float()
    y, mean, rstd = fg.layer_norm(x.cuda())
    y64, mu64, r64 = forward64(x.double(), None, None)
    assert rel(rstd, r64) <= 1e-6
    assert rel(y, y64) <= 1000 * 2.0 ** -22


def test_constant_rows_and_non_finite_values(fg):
    x = torch.ones(6, 300)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = -1e30
    x[5] = torch.linspace(-1, 1, 300)
    y, mean, rstd = fg.layer_norm(x.cuda())
    y = y.cpu()
    assert torch.all(y[0] == 0) and torch.all(y[1] == 0)
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    assert torch.isfinite(y[5]).all()
    assert rel(y[5], forward64(x[5:].double(), None, None)[0][0]) <= tol("f32")


def test_no_rows(fg):
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, mean, rstd = fg.layer_norm(x, w, w)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = fg.layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_same_bits_again_and_on_another_stream(fg):
    x, dy = rand(1, 4099, 1000).bfloat16().cuda(), rand(2, 4099, 1000).bfloat16().cuda()
    w = rand(3, 1000).float().cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    runs = []
    for s in (None, side, None):
        y, mean, rstd = fg.layer_norm(x, w, w, stream=s)
        runs.append((y,) + fg.layer_norm_backward(dy, x, w, mean, rstd, stream=s))
        torch.cuda.synchronize()
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_captures_into_a_graph(fg):
    x, w = rand(1, 40, 512).float().cuda(), rand(2, 512).float().cuda()
    dy = rand(3, 40, 512).float().cuda()
    fg.layer_norm_backward(dy, x, w, *fg.layer_norm(x, w, w)[1:])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, mean, rstd = fg.layer_norm(x, w, w)
        grads = fg.layer_norm_backward(dy, x, w, mean, rstd)
    x.copy_(rand(7, 40, 512))
    graph.replay()
    torch.cuda.synchronize()
    want = fg.layer_norm(x, w, w)
    assert torch.equal(y, want[0])
    assert all(torch.equal(a, b) for a, b in zip(grads, fg.layer_norm_backward(dy, x, w, *want[1:])))


def test_refusals(fg):
    x = torch.zeros(4, 8, device="cuda")
    with pytest.raises(TypeError):
        fg.layer_norm(x.int())
    with pytest.raises(ValueError):
        fg.layer_norm(x.cpu())
    with pytest.raises(ValueError):
        fg.layer_norm(x, torch.ones(7, device="cuda"))
    with pytest.raises(TypeError):
        fg.layer_norm(x, torch.ones(8, device="cuda"), torch.ones(8, device="cuda").half())
    with pytest.raises(fg.FFTError):
        fg.layer_norm(x, torch.ones(8, device="cuda").half())  # 16-bit weight of fp32 rows
    with pytest.raises(fg.FFTError):
        fg.layer_norm(x, eps=-1.0)
    with pytest.raises(ValueError):
        fg.layer_norm(x, out=torch.zeros(4, 9, device="cuda")[:, :8])
    y, mean, rstd = fg.layer_norm(x)
    with pytest.raises(ValueError):
        fg.layer_norm_backward(x[:3], x, None, mean, rstd)
    with pytest.raises(ValueError):
        fg.layer_norm_backward(x, x, None, mean[:3], rstd)
