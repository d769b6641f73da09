"""Binding of the attention over the cache: numbers that do not fit the C ABI's 32 bits, and
queries of a wrong rank, on the host with stand-ins for GPU tensors."""
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
from tests.test_abi_heads_kv import I32, MB, T_BF, U8, Stand, held_cache

MOST = 2 ** 31 - 1


@pytest.fixture
def calls(monkeypatch):
    """The arguments of each nq_kv_attention, which is not made."""
    made, real = [], nq.lib()

    class Recorder:
        def __getattr__(self, name):
            return (lambda *args: made.append(args) or 0) if name == "nq_kv_attention" else getattr(real, name)
    monkeypatch.setattr(nq, "lib", lambda: Recorder())
    monkeypatch.setattr(nq, "_on_stream", lambda device, stream, call: call(0))
    return made


def attend(**kw):
    q = Stand((2, 4, 64), T_BF)
    return nq.kv_attention_into(q, held_cache(), Stand((2, 3), I32), Stand((2,), I32), q, Stand((64 * MB,), U8), **kw)


@pytest.mark.parametrize("given", [0, 1, 48, MOST, MOST + 1, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 70])
def test_a_window_or_length_beyond_32_bits_stays_the_widest(calls, given):
    attend(window=given)
    attend(max_length=given)
    assert calls[0][9] == calls[1][8] == min(given, MOST)
    assert calls[0][8] == calls[1][9] == 0


@pytest.mark.parametrize("given", [-1, -2 ** 31, -2 ** 32, -2 ** 32 + 5])
def test_below_zero_is_refused(calls, given):
    for kw in (dict(window=given), dict(max_length=given)):
        with pytest.raises(nq.NQError):
            attend(**kw)
    assert not calls

def test_queries_of_a_wrong_rank_are_refused(calls, monkeypatch):
    monkeypatch.setattr(nq, "new_kv_workspace", lambda B, q_heads, cache: Stand((64 * MB,), U8))
    monkeypatch.setattr(nq, "_like", lambda t, dtype=None: t)
    for shape in ((), (256,), (2, 256), (1, 2, 4, 64)):
        with pytest.raises(nq.NQError):
            nq.kv_attention(Stand(shape, T_BF), held_cache(), Stand((2, 3), I32), Stand((2,), I32))
    assert not calls
