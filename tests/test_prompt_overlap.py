"""Outputs of the prompt path that share memory with inputs or with one another are refused
before any launch. Addresses here are numbers that no refused call looks at."""
import ctypes

import pytest

from frame_level_delta_b200 import vda as V

GB = 1 << 30


def _at(i, off=0):
    """The i-th of many places far apart."""
    return ctypes.c_void_p((i + 1) * GB + off)


T, N, H, d = 10, 2, 4, 64
ROW = H * d
TOK = T * ROW * 2
STATE = N * H * d * d * 4


def _attention(**at):
    """All apart, but for ``at``."""
    p = {n: _at(i) for i, n in enumerate(("Q", "K", "V", "cu_q", "cu_k", "k_len", "O", "lse", "dO", "dQ", "dK", "dV", "ws"))}
    p["k_len"] = None
    p.update(at)
    return V.vda_attention_config(N, H, H, d, T, T, ROW, ROW, ROW, ROW, 0.1), p


@pytest.mark.parametrize("out,into", [
    ("O", ("Q", 0)), ("O", ("K", 0)), ("O", ("V", 0)), ("O", ("V", TOK - 16)), ("O", ("Q", 16 - TOK)), ("lse", ("O", 64)),
    ("lse", ("Q", 16)), ("O", ("K", ROW * 2))])
def test_attention(out, into):
    name, off = into
    at = {n: i for i, n in enumerate(("Q", "K", "V", "cu_q", "cu_k", "k_len", "O", "lse"))}
    c, p = _attention(**{out: _at(at[name], off)})
    args = [p[n] for n in ("Q", "K", "V", "cu_q", "cu_k", "k_len", "O", "lse", "ws")]
    assert V.lib().vda_causal_attention(ctypes.byref(c), *args, 1 << 40, None) == 1


@pytest.mark.parametrize("out,into", [
    ("dQ", "Q"), ("dQ", "dO"), ("dK", "K"), ("dV", "V"), ("dV", "O"), ("dK", "dV"), ("dQ", "dK"), ("dK", "lse")])
def test_attention_backward(out, into):
    c, p = _attention()
    p[out] = ctypes.c_void_p(p[into].value + 16)
    args = [p[n] for n in ("Q", "K", "V", "O", "dO", "lse", "cu_q", "cu_k", "k_len", "dQ", "dK", "dV", "ws")]
    assert V.lib().vda_causal_attention_backward(ctypes.byref(c), *args, 1 << 40, None) == 1


NAMES = ("Q", "K", "V", "dO", "g", "cu", "S0", "dS", "O", "S", "dQ", "dK", "dV", "dS0", "ws")


def _decay(T=T):
    return V.vda_decay_config(N, H, d, T, ROW, ROW, ROW, ROW, 1.0), {n: _at(i) for i, n in enumerate(NAMES)}


@pytest.mark.parametrize("out,into,off", [
    ("O", "Q", 0), ("O", "K", 0), ("O", "V", 0), ("S", "S0", 16), ("S", "S0", -STATE + 16), ("S", "O", 0), ("O", "S0", STATE - 16)])
def test_decay(out, into, off):
    c, p = _decay()
    p[out] = ctypes.c_void_p(p[into].value + off)
    args = [p[n] for n in ("Q", "K", "V", "g", "cu", "S0", "O", "S", "ws")]
    assert V.lib().vda_decay_attention(ctypes.byref(c), *args, 1 << 40, None) == 1


@pytest.mark.parametrize("out,into,off", [("O", "Q", 0), ("O", "V", 128), ("O", "S", 0), ("S", "K", 16)])
def test_decay_step(out, into, off):
    c, p = _decay(T=N)
    p[out] = ctypes.c_void_p(p[into].value + off)
    args = [p[n] for n in ("Q", "K", "V", "g", "S", "O")]
    assert V.lib().vda_decay_attention_step(ctypes.byref(c), *args, None) == 1


@pytest.mark.parametrize("out,into,off", [
    ("dQ", "dO", 0), ("dQ", "dK", 16), ("dK", "K", 0), ("dV", "V", 0), ("dS0", "S0", 16), ("dS0", "dS", 0), ("dS0", "dV", 0),
    ("dV", "S0", 0)])
def test_decay_backward(out, into, off):
    c, p = _decay()
    p[out] = ctypes.c_void_p(p[into].value + off)
    args = [p[n] for n in ("Q", "K", "V", "dO", "g", "cu", "S0", "dS", "dQ", "dK", "dV", "dS0", "ws")]
    assert V.lib().vda_decay_attention_backward(ctypes.byref(c), *args, 1 << 40, None) == 1
