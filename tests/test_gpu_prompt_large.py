"""The prompt path where elements lie more than 2^32 bytes and 2^31 elements from their tensor's
start: caches, rows of gradients, and rows far apart."""
import numpy as np
import pytest
import torch

from frame_level_delta_b200 import vda as V
from oracle import prompt_oracle as po
from tests.prompt_cases import bounded, f64, rand, rand32, ranges, slopes, starts

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROWS = (1 << 21) + 3000  # x 1024 elements


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    V.lib()


@pytest.fixture(autouse=True)
def _no_timeout():
    yield
    assert V.sequence_poll() == V.VDA_OK
    torch.cuda.empty_cache()


def _far(t, rows=ROWS):
    """t as the last rows of a tensor of ``rows``; what lies before is not initialised."""
    x = torch.empty(rows, *t.shape[1:], dtype=t.dtype, device=DEV)
    x[rows - t.shape[0]:] = t.to(DEV)
    return x


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("tokens", [1, 70])
def test_a_cache_beyond_32_bits(tokens):
    """Two rooms: one from the tensor's start, with its first 500 slots filled, one at its end."""
    Hq, Hkv, d = 16, 8, 128
    nk = [500, 2900]
    Q = rand(231, 2 * tokens, Hq, d, scale=1.5)
    K, Vv = rand(232, sum(nk), Hkv, d), rand(233, sum(nk), Hkv, d)
    ref = po.causal_attention(f64(Q), f64(K), f64(Vv), ranges([tokens] * 2), ranges(nk), d ** -0.5)
    k, v = _far(K[500:]), _far(Vv[500:])
    k[:500], v[:500] = K[:500].to(DEV), Vv[:500].to(DEV)
    O = V.causal_attention(Q.to(DEV), k, v, starts([tokens] * 2, DEV), cu_k=_i32(0, ROWS - 2900, ROWS), k_len=_i32(*nk))
    bounded(f64(O), ref["O"], ref["abs_O"], "O")


def test_gradients_beyond_32_bits():
    H, d, lens = 8, 128, [200, 130]
    T = sum(lens)
    Q, K, Vv, dO = (rand(241 + i, T, H, d, scale=1.5 if i == 0 else 1.0) for i in range(4))
    ref = po.causal_attention(f64(Q), f64(K), f64(Vv), ranges(lens), ranges(lens), d ** -0.5, f64(dO))
    cu = _i32(ROWS - T, ROWS - 130, ROWS)
    q, k, v, g = (_far(t) for t in (Q, K, Vv, dO))
    O, lse = V.causal_attention(q, k, v, cu, return_lse=True)
    bounded(f64(O[-T:]), ref["O"], ref["abs_O"], "O")
    r = V.causal_attention_backward(q, k, v, O, g, lse, cu)
    for n in ("dQ", "dK", "dV"):
        bounded(f64(r[n][-T:]), ref[n], ref["abs_" + n], n)


def test_decay_attention_beyond_32_bits():
    H, d, lens = 8, 128, [700, 130]
    T, N = sum(lens), 2
    Q, K, Vv, dO = rand(251, T, H, d, unit=True), rand(252, T, H, d, unit=True), rand(253, T, H, d), rand(254, T, H, d)
    S0, dS, ld = rand32(255, N, H, d, d), rand32(256, N, H, d, d), slopes(H)
    ref = po.decay_attention(f64(Q), f64(K), f64(Vv), f64(ld), ranges(lens), f64(S0), 1.0, f64(dO), f64(dS))
    cu = _i32(ROWS - T, ROWS - 130, ROWS)
    q, k, v, g = (_far(t) for t in (Q, K, Vv, dO))
    O, S = V.decay_attention(q, k, v, ld.to(DEV), cu, S0=S0.to(DEV))
    bounded(f64(O[-T:]), ref["O"], ref["abs_O"], "O")
    assert (np.abs(f64(S) - ref["S"]) <= 2.0 ** -18 * ref["abs_S"] + 1e-30).all()
    r = V.decay_attention_backward(q, k, v, g, ld.to(DEV), cu, S0=S0.to(DEV), dS=dS.to(DEV))
    for n in ("dQ", "dK", "dV"):
        bounded(f64(r[n][-T:]), ref[n], ref["abs_" + n], n)


def test_rows_far_apart():
    """300 rows of 2^24 elements' distance: one head of a tensor of very many."""
    H, d, T, apart = 1, 64, 300, 1 << 24
    hold = torch.empty(T, apart, dtype=torch.bfloat16, device=DEV)
    Q, K, Vv, dO = (rand(261 + i, T, H, d, unit=i < 2) for i in range(4))
    at = [hold[:, 64 * i:64 * i + d].view(T, H, d) for i in range(5)]
    for x, t in zip(at, (Q, K, Vv, dO)):
        x.copy_(t)
    q, k, v, g, O = at
    cu, ld = starts([T], DEV), slopes(H).to(DEV)
    a = [t.to(DEV) for t in (Q, K, Vv, dO)]
    want, lse = V.causal_attention(*a[:3], cu, return_lse=True)
    V.causal_attention(q, k, v, cu, O=O)
    assert torch.equal(O, want)
    r, w = V.causal_attention_backward(q, k, v, O, g, lse, cu), V.causal_attention_backward(*a[:3], want, a[3], lse, cu)
    assert all(torch.equal(r[n], w[n]) for n in w)
    want, _ = V.decay_attention(*a[:3], ld, cu)
    V.decay_attention(q, k, v, ld, cu, O=O)
    assert torch.equal(O, want)
    r, w = V.decay_attention_backward(q, k, v, g, ld, cu), V.decay_attention_backward(*a, ld, cu)
    assert all(torch.equal(r[n], w[n]) for n in w)
