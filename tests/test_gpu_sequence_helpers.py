"""What the tensor helpers of the sequence-model operators do around the
kernels: streams, rows that belong to no sequence, tensors changed in place.
"""
import pytest

torch = pytest.importorskip("torch")
import delta_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


def test_strided_vectors_on_a_stream(fg):
    # the copies of weight and bias belong to the call's stream: work that is still under way on the
    # current one (which does not touch the inputs) must not hold them back
    x, w, dy = torch.randn(64, 512, device="cuda"), torch.randn(1024, device="cuda"), torch.randn(64, 512, device="cuda")
    b = torch.randn(1024, device="cuda")
    want = fg.layer_norm(x, w[::2].contiguous(), b[::2].contiguous())
    grads = fg.layer_norm_backward(dy, x, w[::2].contiguous(), *want[1:])
    busy, side = torch.randn(8192, 8192, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(8):
            busy @ busy
        got = fg.layer_norm(x, w[::2], b[::2], stream=side)
        back = fg.layer_norm_backward(dy, x, w[::2], *want[1:], stream=side)
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert all(torch.equal(p, q) for p, q in zip(back, grads))
        torch.cuda.synchronize()


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offsets", [[10, 70, 70, 150], [0, 130], [200], [0, 0, 0]])
def test_rows_of_no_sequence_are_zero(fg, kind, offsets):
    args = [t[0].cuda() for t in ref.inputs(16, 1, 200, 1, 2, 40, 64, kind)]
    do = torch.randn(200, 2, 64, device="cuda").to(kind)
    at = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    for _ in range(2):
        # memory that the allocator gives out again is full of these
        junk = [torch.full((n,), float("nan"), device="cuda") for n in (200 * 2, 200 * 2, 200 * 40, 200 * 128, 200 * 64, 200 * 20)]
        del junk
        rows = [fg.delta_rule(*args, offsets=at)[0], *fg.delta_rule_backward(do, *args, offsets=at)[:5]]
        for t in rows:
            assert not t[:offsets[0]].any() and not t[offsets[-1]:].any()
            assert t.isfinite().all()


def raises_for_a_change(make, change):
    """Whether autograd notices that `change` overwrites what a product keeps for its gradient."""
    a = make().requires_grad_()
    kept = a * 1.0
    y = (kept * kept).sum()
    change(kept.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_autograd_notices_tensors_changed_in_place(fg):
    ones = lambda *shape: lambda: torch.ones(*shape, device="cuda")  # noqa: E731
    other = torch.ones(8, device="cuda")
    raises_for_a_change(ones(8), lambda t: fg.clip_grad_norm([t], 0.5))
    raises_for_a_change(ones(8), lambda t: fg.clip_grad_norm([other], 0.5, out=[t]))
    raises_for_a_change(ones(4, 8), lambda t: fg.layer_norm(torch.ones(4, 8, device="cuda"), out=t))
    args = [t.cuda() for t in ref.inputs(17, 2, 3, 1, 2, 16, 24)]
    raises_for_a_change(ones(2, 2, 16, 24), lambda t: fg.delta_rule_step(*args, t))
    pool = torch.zeros(2, 2, 16, 24, device="cuda")
    raises_for_a_change(ones(2, 3, 2, 24), lambda t: fg.delta_rule_step(*args, pool, out=t))
    raises_for_a_change(ones(2, 3, 2, 24), lambda t: fg.delta_rule(*args, out=t))
