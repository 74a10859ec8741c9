"""The 2-norm limits of the prompt path: what the kernels round stays below them, small
mistakes do not. Mistakes are made in the oracle's inputs or results; no GPU is needed."""
import numpy as np
import pytest
import torch

from oracle import prompt_oracle as po
from tests import prompt_norms as pn
from tests.prompt_cases import f64, rand, rand32, slopes


def _bf(x):
    return f64(torch.from_numpy(np.ascontiguousarray(x)).float().to(torch.bfloat16))


def _attention(n, d=64, nq=None, seed=1):
    nq = n if nq is None else nq
    return [f64(rand(seed + i, m, d, scale=1.5 if i == 0 else 1.0)) for i, m in enumerate((nq, n, n, nq))]


@pytest.mark.parametrize("nq,nk", [(300, 300), (8, 4000)])
def test_rounded_weights_stay_below_and_mistakes_do_not(nq, nk):
    q, k, v, do = _attention(nk, nq=nq)
    s = 64 ** -0.5
    r = po.attention_sequence(q, k, v, s, do)
    sq = pn.attention_squares(q, k, v, s, do)
    x = s * (q @ k.T)
    see = np.arange(nk) <= (nk - nq + np.arange(nq))[:, None]
    p = np.where(see, np.exp(x - np.where(see, x, -np.inf).max(1, keepdims=True)), 0.0)
    l = p.sum(1, keepdims=True)
    o = _bf(_bf(p) @ v / l)
    ds = p / l * (do @ v.T - (do * o).sum(1, keepdims=True))
    lim = {n: pn.limit(sq[n], r[m], r["abs_" + m], nk) for n, m in (("O", "o"), ("dQ", "dq"), ("dK", "dk"), ("dV", "dv"))}
    for n, m, got in (("O", "o", o), ("dQ", "dq", _bf(s * _bf(ds) @ k)), ("dK", "dk", _bf(s * _bf(ds).T @ q)),
                      ("dV", "dv", _bf(_bf(p / l).T @ do))):
        assert pn.off(got, r[m]) <= lim[n], n
        assert pn.off(1.01 * r[m], r[m]) > lim[n], n
        assert pn.off(r[m] + 0.01 * r[m].std(), r[m]) > lim[n], n
    # one block of 16 value rows missing from a long row
    w = v.copy()
    w[nk // 2:nk // 2 + 16] = 0
    assert pn.off(po.attention_sequence(q, k, w, s)["o"], r["o"]) > lim["O"]


def test_rounded_states_stay_below_and_mistakes_do_not():
    n, d, chunk = 300, 64, 128
    q, k, v, do = (f64(rand(11 + i, n, 1, d, unit=i < 2)) for i in range(4))
    S0, dS = f64(rand32(15, 1, 1, d, d)), f64(rand32(16, 1, 1, d, d))
    g = f64(slopes(4)[2:3])
    ref = po.decay_attention(q, k, v, g, [(0, n)], S0, 1.0, do, dS)
    sq = pn.decay(q, k, v, g, [(0, n)], S0, 1.0, do, dS)
    a, X, out = np.exp(g[0]), S0[0, 0], np.zeros((n, d))
    for lo in range(0, n, chunk):
        hi = min(n, lo + chunk)
        e = np.arange(hi - lo)
        w = np.where(e[None, :] <= e[:, None], a ** np.maximum(e[:, None] - e, 0.0), 0.0)
        x, y, z = q[lo:hi, 0], k[lo:hi, 0], v[lo:hi, 0]
        out[lo:hi] = _bf(_bf(w * (x @ y.T)) @ z + (a ** (e + 1))[:, None] * (x @ _bf(X).T))
        X = a ** (hi - lo) * X + ((a ** (hi - lo - 1 - e))[:, None] * z).T @ y
    for name in ("O", "dQ", "dK", "dV"):
        lim = pn.limit(sq[name], ref[name], ref["abs_" + name], chunk)
        assert lim < 6e-3 * np.linalg.norm(ref[name])
        assert pn.off(1.01 * ref[name], ref[name]) > lim
        if name == "O":
            assert pn.off(out, ref["O"][:, 0]) <= lim


def test_squares_agree_with_the_definition():
    """With one token to a chunk every term is a state's or a token's own: the squares of the
    reverse passes are those of the forward pass on reversed tokens."""
    n, d = 5, 3
    r = np.random.default_rng(0)
    q, k, v, do = (r.standard_normal((n, 1, d)) for _ in range(4))
    S0, dS = r.standard_normal((2, 1, 1, d, d))
    g = np.array([-0.3])
    sq = pn.decay(q, k, v, g, [(0, n)], S0, 0.7, do, dS, chunk=1)
    a = np.exp(g[0])
    D = dS[0, 0]
    for t in range(n - 1, -1, -1):
        own = 0.7 * np.outer(do[t, 0], q[t, 0])
        np.testing.assert_allclose(sq["dV"][t, 0], (0.7 * (k[t, 0] @ q[t, 0]) * do[t, 0]) ** 2 + D ** 2 @ k[t, 0] ** 2)
        np.testing.assert_allclose(sq["dK"][t, 0], (0.7 * (v[t, 0] @ do[t, 0]) * q[t, 0]) ** 2 + (D ** 2).T @ v[t, 0] ** 2)
        D = a * (D + own)
