"""GPU gradient norm and clipping against 64-bit sums.

Tolerances, fixed before the first run: the norm is a sum of positive terms,
fp32 over groups of 16 bytes (at most 8 terms: 8 * 2^-24) and fp64 beyond,
halved by the root and rounded once to fp32: 8 * 2^-24.  A clipped value is
one product with the rounded factor and one rounding to its type of p bits:
2^-p plus 8 * 2^-24 of its own size.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f64": torch.float64, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float64: 2.0 ** -53, torch.bfloat16: 2.0 ** -8,
            torch.float16: 2.0 ** -11}
FP32 = 8 * 2.0 ** -24


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


def rand(seed, n):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(n))


def norm64(ts):
    return float(torch.sqrt(sum((t.double() ** 2).sum() for t in ts)))


def check(fg, grads, max_norm, eps=1e-6):
    before = [t.clone() for t in grads]
    n = norm64([t.cpu() for t in grads])
    out = [torch.full_like(t, 7) for t in grads]
    norm = fg.clip_grad_norm(grads, max_norm, out=out, eps=eps)
    assert norm.dtype == torch.float32 and norm.shape == ()
    assert abs(float(norm) - n) <= FP32 * n
    assert float(fg.grad_norm(grads)) == float(norm)
    f = min(1.0, max_norm / (n + eps))
    for t, o, b in zip(grads, out, before):
        assert torch.equal(t, b)
        want = b.double().cpu() * f
        small = 6e-8 if t.dtype == torch.float16 else 1e-38  # below: fewer significand bits
        bound = (HALF_ULP[t.dtype] + FP32 * (t.dtype != torch.float64 or 1)) * want.abs() + small
        assert bool(((o.double().cpu() - want).abs() <= bound).all())
    again = fg.clip_grad_norm(grads, max_norm, eps=eps)  # in place
    assert float(again) == float(norm)
    assert all(torch.equal(t, o) for t, o in zip(grads, out))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
@pytest.mark.parametrize("sizes", [(1,), (3, 5), (16384,), (16385, 1, 16383), (100003, 7, 65536),
                                   (1 << 21, 9)])
def test_sizes(fg, kind, max_norm, sizes):
    check(fg, [rand(i, n).to(TYPES[kind]).cuda() for i, n in enumerate(sizes)], max_norm)


def test_mixed_types_and_empty_tensors(fg):
    kinds = list(TYPES.values())
    ts = [rand(i, n).to(kinds[i % 4]).cuda() for i, n in enumerate([0, 10, 300, 0, 0, 70001, 5, 0])]
    check(fg, ts, 1.0)
    check(fg, [torch.empty(0, device="cuda")] * 3, 1.0)


@pytest.mark.parametrize("count", [72, 73, 960, 961, 2000])
def test_many_tensors(fg, count):
    # around the sizes of the argument tables, and more than one launch's table
    rng = np.random.default_rng(count)
    check(fg, [rand(i, int(rng.integers(0, 400))).float().cuda() for i in range(count)], 2.0)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_unaligned_views(fg, kind):
    base, obase = rand(1, 50000).to(TYPES[kind]).cuda(), torch.zeros(50000, dtype=TYPES[kind]).cuda()
    grads = [base[1:20000], base[20007:40000], base[40001:40004]]
    outs = [obase[5:20004], obase[20007:40000], obase[49997:50000]]
    n = norm64([t.cpu() for t in grads])
    norm = fg.clip_grad_norm(grads, 1.0, out=outs)
    assert abs(float(norm) - n) <= FP32 * n
    for t, o in zip(grads, outs):
        assert torch.equal(o, (t.float() * np.float32(1.0 / (n + 1e-6))).to(t.dtype)) or float(
            (o.double() - t.double() / (n + 1e-6)).abs().max()) <= 2 * HALF_ULP[t.dtype] * float(
                t.double().abs().max()) / n
    assert not obase[:5].any() and not obase[20004:20007].any() and not obase[40000:49997].any()


def test_squares_beyond_fp32(fg):
    # 1e25 squared overflows fp32, 1e-30 squared vanishes in it.
    check(fg, [1e25 * rand(1, 5000).float().cuda()], 1.0)
    check(fg, [1e-30 * rand(2, 5000).float().cuda()], 1.0, eps=0.0)
    ts = [1e-30 * rand(2, 64).float().cuda(), torch.zeros(64, device="cuda")]
    assert abs(float(fg.grad_norm(ts)) - norm64([t.cpu() for t in ts])) <= FP32 * norm64([t.cpu() for t in ts])


def test_non_finite(fg):
    ts = [rand(1, 100).float().cuda(), rand(2, 100).float().cuda()]
    ts[0][3] = float("inf")
    out = [torch.empty_like(t) for t in ts]
    assert float(fg.clip_grad_norm(ts, 1.0, out=out)) == float("inf")
    assert not out[1].any() and torch.isnan(out[0][3]) and not out[0][4:].any()
    ts[1][5] = float("nan")
    assert np.isnan(float(fg.clip_grad_norm(ts, 1.0, out=out)))
    assert torch.isnan(out[0]).all() and torch.isnan(out[1]).all()


def test_same_bits_again_on_another_stream_and_in_a_graph(fg):
    ts = [rand(i, 100000 + i).bfloat16().cuda() for i in range(5)]
    out = [torch.empty_like(t) for t in ts]
    torch.cuda.synchronize()
    norms = []
    for s in (None, torch.cuda.Stream(), None):
        norms.append(fg.clip_grad_norm(ts, 1.0, out=out, stream=s))
        torch.cuda.synchronize()
    assert len({float(n) for n in norms}) == 1
    first = [o.clone() for o in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = fg.clip_grad_norm(ts, 1.0, out=out)
    for o in out:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert float(norm) == float(norms[0]) and all(torch.equal(a, b) for a, b in zip(out, first))


def test_refusals(fg):
    t = torch.zeros(8, device="cuda")
    for bad in ([], ):
        with pytest.raises(ValueError):
            fg.clip_grad_norm(bad, 1.0)
    with pytest.raises(TypeError):
        fg.grad_norm([t.int()])
    with pytest.raises(ValueError):
        fg.grad_norm([t.cpu()])
    with pytest.raises(ValueError):
        fg.grad_norm([torch.zeros(4, 4, device="cuda").t()])
    with pytest.raises(ValueError):
        fg.clip_grad_norm([t], 1.0, out=[t[:4]])
    with pytest.raises(ValueError):
        fg.clip_grad_norm([t], 1.0, out=[t.half()])
    with pytest.raises(fg.FFTError):
        fg.clip_grad_norm([t], -1.0)
    with pytest.raises(fg.FFTError):
        fg.clip_grad_norm([t], float("nan"))
