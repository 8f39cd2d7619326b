"""The waits inside the kernels of the linear recurrence and the cross entropy of a
linear layer run out: a barrier of the first block expects one arrival more than
will come (FFT_OPT_STARVED_WAIT).  The call ends, the device status word says so,
and the next call on the context is right.  Nothing is read or written out of
place meanwhile: copies, maps and products that are on their way land before
their block leaves."""
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


# tiles of tokens x words, of words x few tokens; one tile for a pair of blocks and many; three parts of fp32 operands
@pytest.mark.parametrize("barrier", [1, 2, 3, 4])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("tokens,vocabulary,dim", [(300, 2100, 1600), (40, 3000, 1600), (3000, 20000, 136)])
def test_cross_entropy(fg, opt, tokens, vocabulary, dim, kind, barrier):
    x, w = torch.randn(tokens, dim, device="cuda").to(TYPES[kind]), 0.1 * torch.randn(vocabulary, dim, device="cuda")
    w, targets = w.to(TYPES[kind]), torch.randint(-1, vocabulary, (tokens,), device="cuda")
    dloss = torch.rand(tokens, device="cuda")
    run = lambda: (lambda loss, lse: (loss, lse, *fg.linear_cross_entropy_backward(dloss, x, w, targets, lse)))(  # noqa: E731
        *fg.linear_cross_entropy(x, w, targets))
    want, stream = run(), torch.cuda.current_stream().cuda_stream
    assert fg.fft_device_status(stream) == fg.FFT_OK
    for call in (lambda: fg.linear_cross_entropy(x, w, targets),
                 lambda: fg.linear_cross_entropy_backward(dloss, x, w, targets, want[1])):
        opt("STARVED_WAIT", barrier)
        call()
        assert fg.fft_device_status(stream) == fg.FFT_ERR_DEVICE_TIMEOUT
        opt("STARVED_WAIT", -1)
        assert fg.fft_device_status(stream) == fg.FFT_OK
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
    assert fg.fft_device_status(stream) == fg.FFT_OK
