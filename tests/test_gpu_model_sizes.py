"""Large calls of the linear recurrence: packed rows whose elements pass 32-bit
indexes, shared by so many sequences that a batch of them would not be taken."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_recurrence import U, backward64, forward64, within  # noqa: E402


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


def test_many_sequences_in_many_rows(fg):
    sequences, tokens, channels = 20000, 2 ** 20, 4096
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    new = lambda: torch.empty(tokens, channels, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x, dy, g = new().normal_(), new().normal_(), new().uniform_(-0.5, 0)
    at = torch.linspace(0, tokens, sequences + 1, device="cuda", dtype=torch.float64).int()
    y, final = fg.linear_recurrence(x, g, offsets=at)
    dx, dg, _, d0 = fg.linear_recurrence_backward(dy, x, g, y, offsets=at)
    for i in (0, 1, 9999, sequences - 1):
        a, b = int(at[i]), int(at[i + 1])
        (want, s, n), end = forward64(x[a:b], g[a:b], None, None)
        within(y[a:b], want, U * (16 * s + 6 * n))
        within(final[i], end[0], U * (16 * end[1] + 6 * end[2]))
        rows, last = backward64(dy[a:b], x[a:b], g[a:b], y[a:b], None, None, None)
        within(dx[a:b], rows[0], rows[1] + 4 * U * rows[0].abs())
        within(dg[a:b], rows[2], rows[3])
        within(d0[i], last[0], last[1])
