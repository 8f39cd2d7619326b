"""What the tensor helpers of the sequence-model operators do around the
kernels.
"""
import pytest

torch = pytest.importorskip("torch")

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
