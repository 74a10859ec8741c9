"""Float64 statement of the prompt path: causal attention over packed sequences with
grouped heads, and linear attention with a decay for each head, with their gradients.

One sequence at a time, from the definitions; shares no code with the library. Beside
each result stand the sums of absolute values that bound what rounding an operand of
its products to bf16 can change (the tests derive their tolerances from them).
"""
import numpy as np


def _seen(nq, nk):
    """[nq, nk]: the last query stands at the last key."""
    return np.arange(nk)[None, :] <= (nk - nq + np.arange(nq))[:, None]


def attention_sequence(q, k, v, scale, do=None):
    """One sequence and head: q [nq, d], k, v [nk, d]. Returns o, lse, and with ``do``
    dq, dk, dv, each with its bound: abs_* is what one relative unit of rounding of
    the probabilities (and of ds, and of o in do.o) can change."""
    nq, nk = len(q), len(k)
    see = _seen(nq, nk)
    x = np.where(see, scale * (q @ k.T), -np.inf)
    any_key = see.any(1)
    m = np.where(any_key, x.max(1, initial=-np.inf), 0.0)
    p = np.where(see, np.exp(x - m[:, None]), 0.0)
    l = p.sum(1)
    p = p / np.where(any_key, l, 1.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(any_key, m + np.log(l), -np.inf)
    r = {"o": p @ v, "lse": lse, "abs_o": p @ np.abs(v)}
    if do is not None:
        D = (do * r["o"]).sum(1)
        abs_D = (np.abs(do) * np.abs(r["o"])).sum(1)
        ds = p * (do @ v.T - D[:, None])
        abs_ds = np.abs(ds) + p * abs_D[:, None]
        r.update(dq=scale * ds @ k, dk=scale * ds.T @ q, dv=p.T @ do,
                 abs_dq=scale * abs_ds @ np.abs(k), abs_dk=scale * abs_ds.T @ np.abs(q), abs_dv=p.T @ np.abs(do))
    return r


def causal_attention(Q, K, V, q_ranges, k_ranges, scale, dO=None):
    """Packed form: Q [Tq, Hq, d], K, V [Tk, Hkv, d]; sequence i's tokens are
    q_ranges[i] = (lo, hi) of Q and k_ranges[i] of K, V. Rows outside stay NaN."""
    G = Q.shape[1] // K.shape[1]
    out = {"O": np.full(Q.shape, np.nan), "lse": np.full(Q.shape[:2], np.nan), "abs_O": np.full(Q.shape, np.nan)}
    if dO is not None:
        for n, t in (("dQ", Q), ("dK", K), ("dV", V)):
            out[n], out["abs_" + n] = np.full(t.shape, np.nan), np.full(t.shape, np.nan)
    for (a, b), (c, d) in zip(q_ranges, k_ranges):
        if dO is not None:
            for n in ("dK", "dV", "abs_dK", "abs_dV"):
                out[n][c:d] = 0.0
        for h in range(Q.shape[1]):
            g = h // G
            r = attention_sequence(Q[a:b, h], K[c:d, g], V[c:d, g], scale, None if dO is None else dO[a:b, h])
            out["O"][a:b, h], out["lse"][a:b, h], out["abs_O"][a:b, h] = r["o"], r["lse"], r["abs_o"]
            if dO is not None:
                for p in ("", "abs_"):
                    out[p + "dQ"][a:b, h] = r[p + "dq"]
                    out[p + "dK"][c:d, g] += r[p + "dk"]
                    out[p + "dV"][c:d, g] += r[p + "dv"]
    return out


def decay_sequence(q, k, v, a, S0, scale, do=None, dS=None):
    """One sequence, all heads, token by token: q, k, v [n, H, d], a [H], S0 [H, d, d].
    abs_* carry the recurrences over absolute values."""
    n, H, d = q.shape
    S, A = S0.copy(), np.abs(S0)
    w = a[:, None, None]
    o, abs_o = np.zeros_like(q), np.zeros_like(q)
    states, abs_states = [], []
    for t in range(n):
        S = w * S + v[t][:, :, None] * k[t][:, None, :]
        A = w * A + np.abs(v[t])[:, :, None] * np.abs(k[t])[:, None, :]
        states.append(S)
        abs_states.append(A)
        o[t] = scale * np.einsum("hvk,hk->hv", S, q[t])
        abs_o[t] = abs(scale) * np.einsum("hvk,hk->hv", A, np.abs(q[t]))
    r = {"o": o, "S": S, "abs_o": abs_o, "abs_S": A}
    if do is None:
        return r
    for x in ("dq", "dk", "dv"):
        r[x], r["abs_" + x] = np.zeros_like(q), np.zeros_like(q)
    D, B = dS.copy(), np.abs(dS)
    for t in range(n - 1, -1, -1):
        D = D + scale * do[t][:, :, None] * q[t][:, None, :]
        B = B + abs(scale) * np.abs(do[t])[:, :, None] * np.abs(q[t])[:, None, :]
        r["dq"][t] = scale * np.einsum("hvk,hv->hk", states[t], do[t])
        r["dk"][t] = np.einsum("hvk,hv->hk", D, v[t])
        r["dv"][t] = np.einsum("hvk,hk->hv", D, k[t])
        r["abs_dq"][t] = abs(scale) * np.einsum("hvk,hv->hk", abs_states[t], np.abs(do[t]))
        r["abs_dk"][t] = np.einsum("hvk,hv->hk", B, np.abs(v[t]))
        r["abs_dv"][t] = np.einsum("hvk,hk->hv", B, np.abs(k[t]))
        D, B = w * D, w * B
    r["dS0"], r["abs_dS0"] = D, B
    return r


def decay_attention(Q, K, V, log_decay, ranges, S0, scale, dO=None, dS=None):
    """Packed form: Q, K, V [T, H, d], S0 (dS) [N, H, d, d]. Rows outside the ranges stay NaN."""
    a = np.exp(log_decay)
    names = ["O"] + ([] if dO is None else ["dQ", "dK", "dV"])
    out = {p + n: np.full(Q.shape, np.nan) for n in names for p in ("", "abs_")}
    states = ["S"] + ([] if dO is None else ["dS0"])
    out.update({p + n: np.zeros(S0.shape) for n in states for p in ("", "abs_")})
    for i, (lo, hi) in enumerate(ranges):
        r = decay_sequence(Q[lo:hi], K[lo:hi], V[lo:hi], a, S0[i], scale, None if dO is None else dO[lo:hi],
                           None if dO is None else dS[i])
        for n in names:
            for p in ("", "abs_"):
                out[p + n][lo:hi] = r[p + ("o" if n == "O" else n.lower())]
        for n in states:
            for p in ("", "abs_"):
                out[p + n][i] = r[p + n]
    return out
