"""CPU checks of the sizes that the embedding, the linear recurrence and the cross
entropy of a linear layer take: what the header admits is not refused, what passes
the kernels' indexes is (no kernel is launched by any call here)."""
import pytest

P = 4096  # an address that is never looked at


@pytest.fixture(scope="module")
def fg(fg_lib):
    return fg_lib


def recurrence(fg, batch, tokens, channels):
    d = fg.RecurrenceDesc(batch, tokens, channels)
    for n in ("x", "g", "beta"):
        setattr(d, n + "_stride", (tokens * channels, channels))
    return d


# 2^20 rows of 4096 channels are 2^32 elements, however many sequences share them
@pytest.mark.parametrize("batch,tokens,channels", [(20000, 2 ** 20, 4096), (2 ** 24, 2 ** 24, 128), (1025, 2 ** 31 - 1, 2 ** 15)])
def test_packed_rows_count_once(fg, batch, tokens, channels):
    d = recurrence(fg, batch, tokens, channels)
    need = fg.fft_linear_recurrence_workspace_bytes(d, 1)
    assert need >= (batch + 1) * 4
    # as far as the workspace: sizes are accepted, nothing is launched
    assert fg.fft_linear_recurrence(d, P, P, P, P, None, P, P, P, need - 1, None) == fg.FFT_ERR_INVALID_ARG
    assert fg.fft_linear_recurrence_backward(d, P, P, P, P, P, P, None, None, P, P, P, P, P, need - 1,
                                             None) == fg.FFT_ERR_INVALID_ARG
    # a batch of so many tokens each is too large
    assert fg.fft_linear_recurrence(d, P, P, P, None, None, P, P, None, 0, None) == fg.FFT_ERR_UNSUPPORTED
    assert fg.fft_linear_recurrence_backward(d, P, P, P, P, P, None, None, None, P, P, P, P, None, 0,
                                             None) == fg.FFT_ERR_UNSUPPORTED
    assert fg.fft_linear_recurrence_step(d, P, P, P, P, P, 5, P, None) == fg.FFT_ERR_UNSUPPORTED
    assert fg.fft_linear_recurrence_workspace_bytes(d, 0) == 0


def test_packed_rows_have_a_limit(fg):
    d = recurrence(fg, 1025, 2 ** 31 - 1, 2 ** 16)
    assert fg.fft_linear_recurrence_workspace_bytes(d, 1) == 0
    assert fg.fft_linear_recurrence(d, P, P, P, P, None, P, P, P, 1 << 40, None) == fg.FFT_ERR_UNSUPPORTED


def test_starved_waits_are_named(fg):
    for barrier in (0, 5):
        assert fg.fft_debug_set_option(fg.FFT_OPT_STARVED_WAIT, barrier) == fg.FFT_ERR_INVALID_ARG
    for value in (1, 4, -1):
        assert fg.fft_debug_set_option(fg.FFT_OPT_STARVED_WAIT, value) == fg.FFT_OK
