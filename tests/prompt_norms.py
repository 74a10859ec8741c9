"""How far the prompt path's results may be from 64 bits in the 2-norm, from the roundings that
the kernels make.

A rounding to bf16 moves a value by at most U of it, and evenly within its half step: rms U /
sqrt(3) of a value just above a power of two, less of all others (0.735 of that where mantissas
are spread evenly in their logarithm, as in products of random values). Roundings of different
values are independent, so a sum of rounded terms is off by an rms of U / sqrt(3) times the root
of the sum of the terms' squares, and a result's own rounding adds its share in squares. Over
the thousand values and more of a case the norm is within a few percent of its rms, which the
0.735 leaves room for. What is fp32 in the kernels is added as it is worst: a weight is off by
less than 2^-17 of it (its exponential 2.6e-6, its logit's sums and scaling 3e-6), a sum in the
tensor cores by 2^-23 of the result for each step of 16 terms.
"""
import numpy as np

from tests.prompt_cases import U

RMS2 = U * U / 3
WEIGHT = 2.0 ** -17
STEP = 2.0 ** -23


def off(got, want):
    return float(np.linalg.norm(got - want))


def limit(squares, want, abs_sum, terms):
    """squares: the sum of the rounded terms' squares, for each value of ``want``; abs_sum the
    sum of the terms' absolute values; terms: how many there are at most."""
    norm = float(np.linalg.norm(want))
    return float(np.sqrt(RMS2 * (squares.sum() + norm ** 2))) + WEIGHT * float(np.linalg.norm(abs_sum)) \
        + STEP * (terms / 16 + 1) * norm


def attention_squares(q, k, v, scale, do=None):
    """One sequence and head: sums of squares for o, and with ``do`` for dq, dk and dv."""
    nq, nk = len(q), len(k)
    see = np.arange(nk)[None, :] <= (nk - nq + np.arange(nq))[:, None]
    x = np.where(see, scale * (q @ k.T), -np.inf)
    m = x.max(1, initial=-np.inf, keepdims=True)
    p = np.where(see, np.exp(x - np.where(np.isfinite(m), m, 0.0)), 0.0)
    p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    o = p @ v
    r = {"O": p ** 2 @ v ** 2}  # the weights
    if do is not None:
        D = (do * o).sum(1)
        ds2 = (p * (do @ v.T - D[:, None])) ** 2
        # D is taken from O as it was returned: with its weights' rounding and its own
        D2 = (do ** 2 * (r["O"] + o ** 2)).sum(1)
        r["dV"] = (p ** 2).T @ do ** 2
        r["dQ"] = scale ** 2 * (ds2 @ k ** 2 + D2[:, None] * (p @ k) ** 2)
        r["dK"] = scale ** 2 * (ds2.T @ q ** 2 + (p ** 2).T @ (D2[:, None] * q ** 2))
    return r


def attention(Q, K, V, q_ranges, k_ranges, scale, dO=None):
    """Packed form of attention_squares; rows outside the sequences are 0."""
    G = Q.shape[1] // K.shape[1]
    out = {"O": np.zeros(Q.shape)}
    if dO is not None:
        out.update(dQ=np.zeros(Q.shape), dK=np.zeros(K.shape), dV=np.zeros(V.shape))
    for (a, b), (c, d) in zip(q_ranges, k_ranges):
        for h in range(Q.shape[1]):
            g = h // G
            r = attention_squares(Q[a:b, h], K[c:d, g], V[c:d, g], scale, None if dO is None else dO[a:b, h])
            out["O"][a:b, h] = r["O"]
            if dO is not None:
                out["dQ"][a:b, h] = r["dQ"]
                out["dK"][c:d, g] += r["dK"]
                out["dV"][c:d, g] += r["dV"]
    return out


def decay_squares(q, k, v, a, X, edges, own):
    """One sequence and head of out_i = sum_{j <= i} a^(i-j) (q_i.k_j) v_j + a^(i+own) X q_i in
    chunks: the weighted pairs within a chunk and the state before it are rounded. X is what
    the tokens find, [channels of v, channels of k]; own = 1 forward; backward (tokens in
    reverse) 0, where X takes its decay when it has left a token."""
    out = np.zeros(v.shape)
    for lo, hi in zip(edges, edges[1:]):
        e = np.arange(hi - lo)
        w = np.where(e[None, :] <= e[:, None], a ** np.maximum(e[:, None] - e, 0.0), 0.0)
        x, y, z = q[lo:hi], k[lo:hi], v[lo:hi]
        f = a ** (e + own)
        out[lo:hi] = (w * (x @ y.T)) ** 2 @ z ** 2 + f[:, None] ** 2 * (x ** 2 @ (X ** 2).T)
        n = hi - lo
        X = a ** n * X + ((a ** (n - own - e))[:, None] * z).T @ y
    return out


def decay(Q, K, V, log_decay, ranges, S0, scale, dO=None, dS=None, chunk=128):
    a = np.exp(log_decay)
    out = {"O": np.zeros(Q.shape)}
    if dO is not None:
        out.update({n: np.zeros(Q.shape) for n in ("dQ", "dK", "dV")})
    for i, (lo, hi) in enumerate(ranges):
        n = hi - lo
        edges = list(range(0, n, chunk)) + [n]
        back = [n - e for e in reversed(edges)]
        for h in range(Q.shape[1]):
            q, k, v = Q[lo:hi, h], K[lo:hi, h], V[lo:hi, h]
            out["O"][lo:hi, h] = scale ** 2 * decay_squares(q, k, v, a[h], S0[i, h], edges, 1)
            if dO is None:
                continue
            g = dO[lo:hi, h]
            out["dQ"][lo:hi, h] = scale ** 2 * decay_squares(g, v, k, a[h], S0[i, h].T, edges, 1)
            out["dK"][lo:hi, h] = decay_squares(v[::-1], scale * g[::-1], q[::-1], a[h], dS[i, h].T, back, 0)[::-1]
            out["dV"][lo:hi, h] = decay_squares(k[::-1], q[::-1], scale * g[::-1], a[h], dS[i, h], back, 0)[::-1]
    return out
