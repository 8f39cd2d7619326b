"""The waits inside the linear recurrence's kernels run out: a barrier of the first
block expects one arrival more than will come (FFT_OPT_STARVED_WAIT).  The call
ends, the device status word says so, and the next call on the context is right.
Nothing is read or written out of place meanwhile: copies and maps that are on
their way land before their block leaves."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


# one long sequence (a cluster shares it), one block per sequence and 128 channels, short sequences; copied by the TMA or by lanes
@pytest.mark.parametrize("barrier", [1, 2, 3, 4])
@pytest.mark.parametrize("kind,gated", [("f32", True), ("bf16", True), ("f16", False)])
@pytest.mark.parametrize("batch,tokens,channels", [(1, 6000, 128), (40, 700, 512), (100, 150, 256), (1, 4000, 45)])
def test_recurrence(fg, opt, batch, tokens, channels, kind, gated, barrier):
    shape = (batch, tokens, channels)
    x, dy = (torch.randn(shape, device="cuda").to(TYPES[kind]) for _ in range(2))
    g = -torch.rand(shape, device="cuda").to(TYPES[kind])
    beta = torch.rand(shape, device="cuda").to(TYPES[kind]) if gated else None
    run = lambda: (  # noqa: E731
        lambda y, h: (y, h, *fg.linear_recurrence_backward(dy, x, g, y, beta=beta, dfinal_state=h)))(
            *fg.linear_recurrence(x, g, beta))
    want, stream = run(), torch.cuda.current_stream().cuda_stream
    y = want[0].clone()
    assert fg.fft_device_status(stream) == fg.FFT_OK
    # tiles come by the TMA where rows lie on 16 bytes, maps go round where blocks share a sequence
    starved = channels % 4 == 0 if barrier <= 2 else batch == 1
    for call in (lambda: fg.linear_recurrence(x, g, beta),
                 lambda: fg.linear_recurrence_backward(dy, x, g, y, beta=beta, dfinal_state=want[1])):
        opt("STARVED_WAIT", barrier)
        call()
        assert fg.fft_device_status(stream) == (fg.FFT_ERR_DEVICE_TIMEOUT if starved else fg.FFT_OK)
        opt("STARVED_WAIT", -1)
        assert fg.fft_device_status(stream) == fg.FFT_OK
        assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(run(), want))
    assert fg.fft_device_status(stream) == fg.FFT_OK
