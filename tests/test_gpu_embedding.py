"""GPU embedding and its gradient against the formulas in 64 bits.

Tolerances, fixed before the first run, per element: a result is rounded once
to its type (half a step of it, relative), after one product by the scale and
a sum of n terms in float, whose every addition may round by 2^-24 of what is
summed so far: (n + 2) 2^-24 of the sum of the terms' sizes.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f64": torch.float64, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


def rand(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)).cuda()


def some_ids(seed, count, rows, padded=True):
    """Frequent and rare rows, and rows that are none."""
    rng = np.random.default_rng(seed)
    ids = np.minimum(np.exp(rng.random(count) * np.log(rows)).astype(np.int64), rows) - 1
    if padded:
        bad = rng.random(count) < 0.15
        ids[bad] = rng.choice([-1, -100, rows, rows + 5, -2 ** 31, 2 ** 31 - 1], bad.sum())
    return torch.from_numpy(ids).cuda()


def half_step(kind):
    return torch.finfo(TYPES[kind]).eps / 2


def unit(kind):
    return 2.0 ** -53 if kind == "f64" else 2.0 ** -24


def lookup64(ids, table, scale):
    there = (ids >= 0) & (ids < table.shape[0])
    return torch.where(there[..., None], table.double()[torch.where(there, ids, 0)] * scale, 0)


def check_gradient(got, dy, ids, rows, scale, kind, tkind, before=None):
    there = (ids >= 0) & (ids < rows)
    at, d = ids[there], dy.double()[there] * scale
    zeros = torch.zeros(rows, dy.shape[-1], dtype=torch.float64, device="cuda")
    want, size = zeros.index_add(0, at, d), zeros.index_add(0, at, d.abs())
    count = torch.zeros(rows, dtype=torch.float64, device="cuda").index_add(0, at, torch.ones_like(at, dtype=torch.float64))
    if before is not None:
        want, size = want + before.double(), size + before.double().abs()
    bound = half_step(tkind) * want.abs() + (count[:, None] + 3) * unit(kind) * size
    if tkind == "f16":
        bound = bound + 2.0 ** -25  # half a step of the smallest
    assert got.dtype == TYPES[tkind] and got.shape == want.shape
    assert ((got.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("tokens,rows,dim", [(1, 1, 1), (1, 5, 8), (3, 2, 7), (33, 40, 16), (70, 9, 100), (257, 300, 33),
                                             (64, 1000, 520), (5, 50, 2048), (2, 9, 4099)])
def test_lookup(fg, kind, tokens, rows, dim):
    table, ids = rand(1, rows, dim).to(TYPES[kind]), some_ids(2, tokens, rows)
    for index in (ids, ids.clamp(-2 ** 31, 2 ** 31 - 1).int()):
        y = fg.embedding(index, table, scale=1.7)
        want = lookup64(ids, table, 1.7)
        assert y.dtype == table.dtype and y.shape == (tokens, dim)
        assert ((y.double() - want).abs() <= (half_step(kind) + 2 * unit(kind)) * want.abs() + 2.0 ** -25).all()
    assert torch.equal(fg.embedding(ids.clamp(0, rows - 1), table), table[ids.clamp(0, rows - 1)])


def test_lookup_shapes_strides_and_out(fg):
    wide = rand(1, 30, 64).float()
    ids = some_ids(2, 24, 30).reshape(2, 3, 4)
    for table in (wide, wide[:, :40], wide[:, 3:35], wide[::2], wide.t(), wide[:, ::2]):
        y = fg.embedding(ids % table.shape[0], table)
        assert torch.equal(y, table[ids % table.shape[0]])
    out = torch.full((2, 3, 4, 64), 7.0, device="cuda")
    assert fg.embedding(ids.transpose(0, 1).transpose(0, 1), wide, out=out) is out
    assert torch.equal(out, lookup64(ids, wide, 1).float())
    assert fg.embedding(ids[:0], wide).shape == (0, 3, 4, 64)
    with pytest.raises(TypeError):
        fg.embedding(ids.float(), wide)
    with pytest.raises(ValueError):
        fg.embedding(ids, wide[0])
    with pytest.raises(ValueError):
        fg.embedding(ids, wide, out=out[..., :32])
    with pytest.raises(ValueError):
        fg.embedding(ids.cpu(), wide)


CASES = [(1, 1, 1), (2, 1, 3), (31, 4, 8), (32, 4, 8), (33, 4, 8), (64, 2, 40), (65, 1, 5), (100, 511, 24), (1000, 512, 17),
         (1025, 513, 64), (3000, 3, 300), (5003, 30011, 33), (9000, 70000, 16), (40000, 20, 24), (20000, 300000, 8), (70001, 500, 24), (300000, 4000, 8)]


@pytest.mark.parametrize("kind,tkind", [("f32", "f32"), ("f64", "f64"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                        ("f16", "f32")])
@pytest.mark.parametrize("tokens,rows,dim", CASES)
def test_gradient(fg, tokens, rows, dim, kind, tkind):
    dy, ids = rand(1, tokens, dim).to(TYPES[kind]), some_ids(2, tokens, rows)
    got = fg.embedding_backward(dy, ids, rows, scale=0.6, dtype=TYPES[tkind])
    check_gradient(got, dy, ids, rows, 0.6, kind, tkind)
    assert torch.equal(got, fg.embedding_backward(dy, ids, rows, scale=0.6, dtype=TYPES[tkind]))  # the same bits
    before = rand(3, rows, dim).to(TYPES[tkind])
    added = before.clone()
    assert fg.embedding_backward(dy, ids, rows, scale=0.6, add_to=added) is added
    check_gradient(added, dy, ids, rows, 0.6, kind, tkind, before)
    untouched = torch.ones(rows, dtype=torch.bool, device="cuda")
    untouched[ids[(ids >= 0) & (ids < rows)]] = False
    assert torch.equal(added[untouched], before[untouched])


@pytest.mark.parametrize("ids", [[-1] * 40, [3] * 100, [3] * 32 + [4] * 32, list(range(64)), [0] * 31 + [1] * 2 + [2] * 95,
                                 [63] * 33 + [64] * 5])
@pytest.mark.parametrize("dim", [8, 9])
def test_runs_and_pieces(fg, ids, dim):
    ids = torch.tensor(ids, device="cuda")
    dy = rand(1, len(ids), dim).float()
    check_gradient(fg.embedding_backward(dy, ids, 64), dy, ids, 64, 1.0, "f32", "f32")


def test_gradient_is_the_lookups(fg):
    # <dy, embed(T)> = <dT, T> for every T: the lookup is linear in the table
    ids, table, dy = some_ids(2, 500, 60), rand(3, 60, 36), rand(4, 500, 36)
    left = (dy * fg.embedding(ids, table, scale=3.0)).sum()
    right = (fg.embedding_backward(dy, ids, 60, scale=3.0) * table).sum()
    assert abs(float(left - right)) <= 1e-12 * 500 * 36


def test_no_tokens(fg):
    dy, ids = torch.empty(0, 12, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    junk = torch.full((9 * 12,), float("nan"), device="cuda")
    del junk
    assert not fg.embedding_backward(dy, ids, 9).any()
    kept = torch.ones(9, 12, device="cuda")
    fg.embedding_backward(dy, ids, 9, add_to=kept)
    assert (kept == 1).all()


def test_strided_gradients_and_refusals(fg):
    wide, ids = rand(1, 90, 64).float(), some_ids(2, 90, 11)
    for dy in (wide[:, :32], wide[:, 5:38], wide[:, ::2], rand(5, 48, 90).float().t()):
        check_gradient(fg.embedding_backward(dy, ids, 11), dy, ids, 11, 1.0, "f32", "f32")
    with pytest.raises(ValueError):
        fg.embedding_backward(wide, ids[:80], 11)
    with pytest.raises(ValueError):
        fg.embedding_backward(wide, ids, 11, add_to=torch.zeros(12, 64, device="cuda"))
    with pytest.raises(TypeError):
        fg.embedding_backward(wide, ids, 11, add_to=torch.zeros(11, 64, device="cuda"), dtype=torch.float64)
    with pytest.raises(fg.FFTError):
        fg.embedding_backward(wide, ids, 11, dtype=torch.bfloat16)
    with pytest.raises(fg.FFTError):
        fg.embedding_backward(wide, ids, 0)


def test_captured_and_replayed(fg):
    ids, dy, table = some_ids(2, 700, 90), rand(1, 700, 40).bfloat16(), rand(4, 90, 40).bfloat16()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for _ in range(2):
            fg.embedding(ids, table), fg.embedding_backward(dy, ids, 90)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, d = fg.embedding(ids, table), fg.embedding_backward(dy, ids, 90)
    for seed in (5, 6):
        ids.copy_(some_ids(seed, 700, 90))
        dy.copy_(rand(seed, 700, 40))
        graph.replay()
        assert torch.equal(y, fg.embedding(ids, table)) and torch.equal(d, fg.embedding_backward(dy, ids, 90))
