"""Calls at the edges of the prompt path's ranges, against the float64 oracle."""
import numpy as np
import pytest
import torch

from frame_level_delta_b200 import vda as V
from oracle import prompt_oracle as po
from tests.prompt_cases import bounded, f64, rand, rand32, ranges, starts

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    V.lib()


@pytest.fixture(autouse=True)
def _no_timeout():
    yield
    assert V.sequence_poll() == V.VDA_OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [-0.4, -1.0, -3.0])
def test_large_values_in_heads_that_forget_fast(g, d):
    """Outputs near 2^32 (keys that meet their own query at 2^6 a channel) where a chunk's
    decay falls far below what fp32 holds. The bounds are relative, so they hold at any size."""
    H, lens = 2, [200, 128]
    T = sum(lens)
    K, Vv, dO = rand(61, T, H, d, scale=64.0), rand(62, T, H, d, scale=1024.0), rand(63, T, H, d, scale=1024.0)
    Q = K.clone()
    S0, dS = rand32(64, len(lens), H, d, d), rand32(65, len(lens), H, d, d)
    ld = torch.full((H,), g)
    ref = po.decay_attention(f64(Q), f64(K), f64(Vv), f64(ld), ranges(lens), f64(S0), 1.0, f64(dO), f64(dS))
    a = [t.to(DEV) for t in (Q, K, Vv)]
    O, _ = V.decay_attention(*a, ld.to(DEV), starts(lens, DEV), S0=S0.to(DEV))
    bounded(f64(O), ref["O"], ref["abs_O"], "O")
    r = V.decay_attention_backward(*a, dO.to(DEV), ld.to(DEV), starts(lens, DEV), S0=S0.to(DEV), dS=dS.to(DEV))
    for n in ("dQ", "dK", "dV"):
        bounded(f64(r[n]), ref[n], ref["abs_" + n], n)


@pytest.mark.parametrize("Hq,Hkv,d", [(2, 2, 64), (4, 2, 128), (3, 1, 128)])
def test_gradients_on_the_diagonal_are_rounded_once(Hq, Hkv, d):
    """Of sequences within one key block, every operand of dQ and dK but O has 16 bits or
    more: next to the gradients' formula on the O that was returned, only the results' own
    rounding is left. What else there is (2^-16 of dS, logits in fp32, about 2^-18 of a
    weight) is below 2^-15, and the rounding's rms above 2^-10: together 1.001 of it in the
    2-norm; one bf16 operand more would give 1.4."""
    lens = [128, 1, 100, 61]
    T, G, s = sum(lens), Hq // Hkv, d ** -0.5
    Q, K, Vv = rand(71, T, Hq, d, scale=1.5), rand(72, T, Hkv, d), rand(73, T, Hkv, d)
    dO, cu = rand(74, T, Hq, d), starts(lens, DEV)
    q, k, v, do = (t.to(DEV) for t in (Q, K, Vv, dO))
    O, lse = V.causal_attention(q, k, v, cu, return_lse=True)
    got = V.causal_attention_backward(q, k, v, O, do, lse, cu)
    Qd, Kd, Vd, Gd, Od = (f64(t) for t in (Q, K, Vv, dO, O))
    want = {"dQ": np.zeros(Qd.shape), "dK": np.zeros(Kd.shape)}
    for lo, hi in ranges(lens):
        for h in range(Hq):
            x = s * Qd[lo:hi, h] @ Kd[lo:hi, h // G].T
            p = np.tril(np.exp(x - x.max(1, keepdims=True)))
            p /= p.sum(1, keepdims=True)
            ds = p * (Gd[lo:hi, h] @ Vd[lo:hi, h // G].T - (Gd[lo:hi, h] * Od[lo:hi, h]).sum(1, keepdims=True))
            want["dQ"][lo:hi, h] = s * ds @ Kd[lo:hi, h // G]
            want["dK"][lo:hi, h // G] += s * ds.T @ Qd[lo:hi, h]
    for n, w in want.items():
        once = np.linalg.norm(f64(torch.from_numpy(w).to(torch.bfloat16)) - w)
        assert np.linalg.norm(f64(got[n]) - w) <= 1.1 * once, n


@pytest.mark.parametrize("Hq,Hkv,d", [(6, 2, 128), (4, 4, 64), (32, 1, 128)])
@pytest.mark.parametrize("N", [8, 40])
def test_few_tokens_on_long_caches(Hq, Hkv, d, N):
    """Some sequences with more tokens than a tile of few rows has, one without any, caches
    that are empty or shorter than the new tokens, NaN in the room behind them."""
    room = 1100
    nq = ([1, 33, 1, 0, 2, 1, 1, 1] if Hq < 32 else [1, 2, 1, 0, 1, 1, 1, 1]) * (N // 8)
    lens = ([1100, 129, 0, 700, 1, 1024, 1099, 513] * (N // 8))
    T = sum(nq)
    tail = 3 if Hq < 32 else 0  # (rows behind count for the choice of form)
    Q, K, Vv = rand(81, T + tail, Hq, d, scale=1.5), rand(82, N * room, Hkv, d), rand(83, N * room, Hkv, d)
    for i, n in enumerate(lens):
        K[i * room + n:(i + 1) * room] = float("nan")
        Vv[i * room + n:(i + 1) * room] = float("nan")
    kr = [(i * room, i * room + n) for i, n in enumerate(lens)]
    ref = po.causal_attention(f64(Q), f64(K), f64(Vv), ranges(nq), kr, d ** -0.5)
    O = torch.full_like(Q, float("nan"), device=DEV)
    _, lse = V.causal_attention(Q.to(DEV), K.to(DEV), Vv.to(DEV), starts(nq, DEV), cu_k=starts([room] * N, DEV),
                                k_len=torch.tensor(lens, dtype=torch.int32, device=DEV), O=O, return_lse=True)
    bounded(f64(O), ref["O"], ref["abs_O"], "O")
    assert np.isnan(f64(O)[T:]).all()
    w, g = ref["lse"][:T], f64(lse)[:T]
    assert np.array_equal(np.isneginf(g), np.isneginf(w))
    ok = np.isfinite(w)
    assert np.abs(g[ok] - w[ok]).max() <= 2.0 ** -11 + 1e-6 * np.abs(w[ok]).max()
