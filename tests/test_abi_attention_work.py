"""C ABI of the attention over the cache: how much work one call may have.  The kernels
count the steps of all sequences in 31 bits: a sequence of n tokens (with a window those
seen) that costs ceil(n / 32) steps and 8 more.  Refusals on the host; a call that is not
refused for its work is told from one that is by its next fault, a q of NULL, so that
nothing is ever launched."""
import ctypes
import os

import pytest

import binary_rank_gemv_packed_amd as nq

FAKE, GB = 0x7F0000000000, 1 << 30
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nq.LIB_PATH):
        from binary_rank_gemv_packed_amd import build
        build.build()
    return nq.lib()


def fault(L, B, tokens, window=0, page=16):
    """The complaint about a call of B sequences of up to `tokens` tokens without q."""
    c = nq.nq_kv_cache(4, 2, 64, page, 0, FAKE)
    width = -(-tokens // page)
    status = L.nq_kv_attention(ctypes.byref(c), B, None, nq.NQ_BF16, 4, FAKE + GB, width, FAKE + 1024 * GB, tokens, window,
                               0.125, FAKE + 1025 * GB, nq.NQ_BF16, FAKE + 1027 * GB, GB, None)
    assert status == nq.NQ_ERR_INVALID_ARG
    return L.nq_last_error().decode()


def seen_steps(tokens, window):
    """Most steps of 32 that a sequence of up to `tokens` tokens touches, by trying its ends."""
    if not window or window >= tokens:
        return -(-tokens // 32)
    return max(-(-n // 32) - (n - window) // 32 for n in range(max(window, tokens - 32), tokens + 1))


EDGES = [(65535, 1048320), (65535, 1048321), (2, 2 ** 30), (63, 1 << 30), (64, (1 << 30) - 256), (64, (1 << 30) - 255),
         (64, 1 << 30), (1000, 68718976), (1000, 68719168), (1000, 68719169), (1, 1 << 30)]


@pytest.mark.parametrize("B,tokens", EDGES)
def test_steps_of_a_call(L, B, tokens):
    fits = B * (-(-tokens // 32) + 8) <= MOST
    assert ("q is NULL" in fault(L, B, tokens)) == fits


@pytest.mark.parametrize("B,window", [(65535, w) for w in (1, 2, 31, 32, 33, 34, 4096, 1048288, 1048289, 1048290, 1048321)] +
                         [(1000, 1 << 20), (64, (1 << 30) - 287), (64, (1 << 30) - 286)])
def test_a_window_bounds_the_steps(L, B, window):
    """What a window hides costs nothing, however long the sequences are."""
    tokens = 1 << 30
    fits = B * (seen_steps(tokens, window) + 8) <= MOST
    assert ("q is NULL" in fault(L, B, tokens, window)) == fits


def test_a_window_wider_than_the_sequences(L):
    assert "q is NULL" in fault(L, 65535, 1048320, window=1 << 30)
    assert "q is NULL" not in fault(L, 65535, 1048321, window=1 << 30)
