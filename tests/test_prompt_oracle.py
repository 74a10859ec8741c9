"""The prompt path's float64 oracle against facts independent of it, and the argument
checks of the prompt path's calls. No test here needs a GPU; no call passes its checks."""
import ctypes

import numpy as np
import pytest
import torch

from frame_level_delta_b200 import vda as V
from oracle import prompt_oracle as po


def _draw(seed, *shapes):
    r = np.random.default_rng(seed)
    return [r.standard_normal(s) for s in shapes]


# ------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("nq,nk", [(1, 1), (5, 5), (3, 9), (7, 4), (2, 0)])
def test_attention_is_a_masked_softmax(nq, nk):
    q, k, v = _draw(0, (nq, 6), (nk, 6), (nk, 6))
    r = po.attention_sequence(q, k, v, 0.7)
    for i in range(nq):
        n = nk - nq + i + 1
        if n <= 0:
            assert (r["o"][i] == 0).all() and np.isneginf(r["lse"][i])
            continue
        x = 0.7 * k[:n] @ q[i]
        w = np.exp(x) / np.exp(x).sum()
        np.testing.assert_allclose(r["o"][i], w @ v[:n], rtol=1e-12)
        np.testing.assert_allclose(r["lse"][i], np.log(np.exp(x).sum()), rtol=1e-12)


def _differences(f, x, up, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        d = np.zeros_like(x)
        d[i] = eps
        g[i] = ((f(x + d) - f(x - d)) * up).sum() / (2 * eps)
    return g


@pytest.mark.parametrize("nq,nk", [(4, 4), (2, 5), (5, 3)])
def test_attention_gradients_against_differences(nq, nk):
    q, k, v, do = _draw(1, (nq, 3), (nk, 3), (nk, 3), (nq, 3))
    r = po.attention_sequence(q, k, v, 0.9, do)
    np.testing.assert_allclose(r["dq"], _differences(lambda x: po.attention_sequence(x, k, v, 0.9)["o"], q, do),
                               atol=1e-7)
    np.testing.assert_allclose(r["dk"], _differences(lambda x: po.attention_sequence(q, x, v, 0.9)["o"], k, do),
                               atol=1e-7)
    np.testing.assert_allclose(r["dv"], _differences(lambda x: po.attention_sequence(q, k, x, 0.9)["o"], v, do),
                               atol=1e-7)


def test_grouped_heads_sum_their_key_gradients():
    Q, K, Vv, dO = _draw(2, (6, 4, 3), (6, 2, 3), (6, 2, 3), (6, 4, 3))
    r = po.causal_attention(Q, K, Vv, [(0, 4), (4, 6)], [(0, 4), (4, 6)], 0.5, dO)
    wide = po.causal_attention(Q, K.repeat(2, 1), Vv.repeat(2, 1), [(0, 4), (4, 6)], [(0, 4), (4, 6)], 0.5, dO)
    np.testing.assert_allclose(r["O"], wide["O"], rtol=1e-12)
    np.testing.assert_allclose(r["dK"], wide["dK"].reshape(6, 2, 2, 3).sum(2), rtol=1e-12)
    np.testing.assert_allclose(r["dV"], wide["dV"].reshape(6, 2, 2, 3).sum(2), rtol=1e-12)


def test_decay_is_a_weighted_sum_over_the_past():
    n, H, d = 7, 2, 3
    q, k, v, S0 = _draw(3, (n, H, d), (n, H, d), (n, H, d), (H, d, d))
    a = np.array([0.9, 0.3])
    r = po.decay_sequence(q, k, v, a, S0, 0.7)
    for h in range(H):
        for t in range(n):
            o = a[h] ** (t + 1) * S0[h] @ q[t, h]
            for j in range(t + 1):
                o = o + a[h] ** (t - j) * (k[j, h] @ q[t, h]) * v[j, h]
            np.testing.assert_allclose(r["o"][t, h], 0.7 * o, rtol=1e-12)
        S = a[h] ** n * S0[h] + sum(a[h] ** (n - 1 - j) * np.outer(v[j, h], k[j, h]) for j in range(n))
        np.testing.assert_allclose(r["S"][h], S, rtol=1e-12)


def test_decay_gradients_against_differences():
    n, H, d = 4, 2, 2
    q, k, v, S0, do, dS = _draw(4, (n, H, d), (n, H, d), (n, H, d), (H, d, d), (n, H, d), (H, d, d))
    a = np.array([0.8, 0.5])

    def loss_of(**kw):
        x = dict(q=q, k=k, v=v, S0=S0)
        x.update(kw)
        r = po.decay_sequence(x["q"], x["k"], x["v"], a, x["S0"], 1.3)
        return np.array((r["o"] * do).sum() + (r["S"] * dS).sum())

    r = po.decay_sequence(q, k, v, a, S0, 1.3, do, dS)
    for n_, x in (("q", q), ("k", k), ("v", v), ("S0", S0)):
        np.testing.assert_allclose(r["d" + n_], _differences(lambda y: loss_of(**{n_: y}), x, 1.0), atol=1e-7)


# ------------------------------------------------------------------ argument checks of the C calls
A = ctypes.c_void_p(1 << 20)  # an aligned address that no refused call looks at
ODD = ctypes.c_void_p((1 << 20) + 2)


def _attn(**kw):
    c = dict(N=2, Hq=4, Hkv=2, d=128, Tq=10, Tk=10, q_row=512, k_row=256, v_row=256, o_row=512, scale=0.1)
    c.update(kw)
    return V.vda_attention_config(*c.values())


def _dec(**kw):
    c = dict(N=2, H=4, d=64, T=10, q_row=256, k_row=256, v_row=256, o_row=256, scale=1.0)
    c.update(kw)
    return V.vda_decay_config(*c.values())


@pytest.mark.parametrize("kw,want", [
    (dict(N=0), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(Tq=-1), 1), (dict(Tk=-1), 1), (dict(scale=0.0), 1),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(d=96), 2),
    (dict(d=32), 2), (dict(Hq=258, Hkv=2, q_row=258 * 128, o_row=258 * 128), 2), (dict(q_row=511), 1),
    (dict(q_row=504), 1), (dict(k_row=248), 1), (dict(v_row=260), 1), (dict(o_row=0), 1), (dict(Tk=1 << 30), 2),
])
def test_attention_configs_are_checked(kw, want):
    c, n = _attn(**kw), ctypes.c_size_t(7)
    L = V.lib()
    assert L.vda_causal_attention_workspace(ctypes.byref(c), ctypes.byref(n)) == want
    assert L.vda_causal_attention_backward_workspace(ctypes.byref(c), ctypes.byref(n)) == want
    assert n.value == 7
    assert L.vda_causal_attention(ctypes.byref(c), A, A, A, A, A, None, A, None, A, 1 << 40, None) == want
    assert L.vda_causal_attention_backward(ctypes.byref(c), *[A] * 6, A, A, None, A, A, A, A, 1 << 40, None) == want


def test_attention_pointers_are_checked():
    c = _attn()
    L = V.lib()
    base = [A, A, A, A, A, None, A, None, A, 1 << 40, None]  # Q K V cu_q cu_k k_len O lse ws bytes stream
    for i in (0, 1, 2, 3, 4, 6):
        x = list(base)
        x[i] = None
        assert L.vda_causal_attention(ctypes.byref(c), *x) == 1
    for i in (0, 1, 2, 6):
        x = list(base)
        x[i] = ctypes.c_void_p((1 << 20) + 8)
        assert L.vda_causal_attention(ctypes.byref(c), *x) == 3
    for i in (3, 4, 5, 7):
        x = list(base)
        x[i] = ODD
        assert L.vda_causal_attention(ctypes.byref(c), *x) == 3
    assert L.vda_causal_attention(None, *base) == 1
    # backward: Q K V O dO lse cu_q cu_k k_len dQ dK dV ws bytes stream
    base = [A] * 8 + [None] + [A] * 4 + [1 << 40, None]
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 9, 10, 11, 12):
        x = list(base)
        x[i] = None
        assert L.vda_causal_attention_backward(ctypes.byref(c), *x) == 1
    x = list(base)
    x[13] = 16
    assert L.vda_causal_attention_backward(ctypes.byref(c), *x) == 4
    x = list(base)
    x[12] = ctypes.c_void_p((1 << 20) + 128)
    assert L.vda_causal_attention_backward(ctypes.byref(c), *x) == 3


def test_split_attention_needs_its_workspace():
    c = _attn(N=1, Tq=1, Tk=100000)
    n = ctypes.c_size_t(0)
    L = V.lib()
    assert L.vda_causal_attention_workspace(ctypes.byref(c), ctypes.byref(n)) == 0 and n.value > 0
    args = [A, A, A, A, A, None, A, None]
    assert L.vda_causal_attention(ctypes.byref(c), *args, None, 0, None) == 1
    assert L.vda_causal_attention(ctypes.byref(c), *args, A, n.value - 1, None) == 4


@pytest.mark.parametrize("kw,want", [
    (dict(N=0), 1), (dict(H=0), 1), (dict(T=-1), 1), (dict(d=128), 1), (dict(d=32), 2), (dict(scale=float("inf")), 1),
    (dict(q_row=255), 1), (dict(k_row=0), 1), (dict(v_row=252), 1), (dict(o_row=8), 1), (dict(T=1 << 30), 2),
    (dict(N=65536), 2),
])
def test_decay_configs_are_checked(kw, want):
    c, n = _dec(**kw), ctypes.c_size_t(7)
    L = V.lib()
    assert L.vda_decay_attention_workspace(ctypes.byref(c), ctypes.byref(n)) == want
    assert L.vda_decay_attention_backward_workspace(ctypes.byref(c), ctypes.byref(n)) == want
    assert L.vda_decay_attention(ctypes.byref(c), *[A] * 8, A, 1 << 40, None) == want
    assert L.vda_decay_attention_backward(ctypes.byref(c), *[A] * 6, None, None, *[A] * 4, A, 1 << 40, None) == want


def test_decay_pointers_are_checked():
    c = _dec()
    L = V.lib()
    base = [A] * 8 + [A, 1 << 40, None]  # Q K V log_decay cu S0 O S ws bytes stream
    for i in (0, 1, 2, 3, 4, 6):
        x = list(base)
        x[i] = None
        assert L.vda_decay_attention(ctypes.byref(c), *x) == 1
    for i in (0, 1, 2, 5, 6, 7):
        x = list(base)
        x[i] = ctypes.c_void_p((1 << 20) + 8)
        assert L.vda_decay_attention(ctypes.byref(c), *x) == 3
    # step: T must be N, the state is required
    args = [A, A, A, A, A, A, None]
    assert L.vda_decay_attention_step(ctypes.byref(_dec(T=3)), *args) == 1
    args[4] = None
    assert L.vda_decay_attention_step(ctypes.byref(_dec(T=2)), *args) == 1
    # backward: dS0 may not be dS or S0
    B = ctypes.c_void_p(1 << 21)
    tail = [A, 1 << 40, None]
    assert L.vda_decay_attention_backward(ctypes.byref(c), *[A] * 6, B, None, A, A, A, B, *tail) == 1
    assert L.vda_decay_attention_backward(ctypes.byref(c), *[A] * 6, None, B, A, A, A, B, *tail) == 1


# ------------------------------------------------------------------ argument checks of the binding
def test_binding_refuses_host_tensors():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    g = torch.zeros(2)
    S = torch.zeros(4, 2, 64, 64)
    with pytest.raises(ValueError, match="CUDA devices"):
        V.causal_attention(q, q, q, cu)
    with pytest.raises(ValueError, match="CUDA devices"):
        V.causal_attention_backward(q, q, q, q, q, torch.zeros(4, 2), cu)
    with pytest.raises(ValueError, match="CUDA devices"):
        V.decay_attention(q, q, q, g, cu)
    with pytest.raises(ValueError, match="CUDA devices"):
        V.decay_attention_step(q, q, q, g, S)
    with pytest.raises(ValueError, match="CUDA devices"):
        V.decay_attention_backward(q, q, q, q, g, cu)
    with pytest.raises(ValueError, match="expected a torch.Tensor"):
        V.causal_attention([1.0], q, q, cu)


def test_binding_checks_rows():
    cpu = torch.device("cpu")
    t = torch.zeros(6, 3, 64, dtype=torch.bfloat16)
    assert V._rows("Q", t, (None, None, None), cpu) == 192
    assert V._rows("Q", torch.zeros(6, 9, 64, dtype=torch.bfloat16)[:, 2:5], (6, 3, 64), cpu) == 576
    assert V._rows("Q", t[:1], (1, 3, 64), cpu) == 192
    for bad, match in ((t.float(), "dtype"), (t[0], "shape"), (t.transpose(1, 2), "contiguous heads"),
                       (t[:, ::2], "contiguous heads"), (t.flip(2)[:, :, ::2], "contiguous heads"),
                       (t.as_strided((6, 3, 64), (100, 64, 1)), "multiple of 8"),
                       (t.as_strided((6, 3, 64), (64, 64, 1)), "not overlap"),
                       (t.as_strided((6, 3, 64), (0, 64, 1)), "not overlap")):
        with pytest.raises(ValueError, match=match):
            V._rows("Q", bad, (None, None, None), cpu)
    with pytest.raises(ValueError, match="shape"):
        V._rows("K", t, (6, 3, 128), cpu)
    for cu in (torch.tensor([0], dtype=torch.int32), torch.tensor(0, dtype=torch.int32), [0, 3]):
        with pytest.raises(ValueError):
            V._starts("cu", cu, cpu)
    with pytest.raises(ValueError, match="dtype"):
        V._starts("cu", torch.tensor([0, 3]), cpu)


@pytest.mark.parametrize("scale", [torch.tensor(0.5), torch.ones(1), np.ones(()), "1"])
def test_binding_takes_numbers_as_scale(scale):
    """A call's checks are remembered by its scale: an object whose value can change is refused."""
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu, g, lse, S = torch.tensor([0, 4], dtype=torch.int32), torch.zeros(2), torch.zeros(4, 2), torch.zeros(4, 2, 64, 64)
    for call in (lambda: V.causal_attention(q, q, q, cu, scale=scale),
                 lambda: V.causal_attention_backward(q, q, q, q, q, lse, cu, scale=scale),
                 lambda: V.decay_attention(q, q, q, g, cu, scale=scale),
                 lambda: V.decay_attention_step(q, q, q, g, S, scale=scale),
                 lambda: V.decay_attention_backward(q, q, q, q, g, cu, scale=scale)):
        with pytest.raises(ValueError, match="scale"):
            call()


def test_binding_takes_any_real_scale():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for scale in (None, 1, 0.5, np.float32(0.5), np.float64(2.0)):
        with pytest.raises(ValueError, match="CUDA devices"):
            V.causal_attention(q, q, q, torch.tensor([0, 4], dtype=torch.int32), scale=scale)
