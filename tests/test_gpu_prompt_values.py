"""Values that must and must not reach a result of the prompt path: NaN behind the keys of a
tile whose warps have few rows or none, against the float64 oracle."""
import numpy as np
import pytest
import torch

from frame_level_delta_b200 import vda as V
from oracle import prompt_oracle as po
from tests.prompt_cases import bounded, f64, rand, ranges, starts

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    V.lib()


@pytest.fixture(autouse=True)
def _no_timeout():
    yield
    assert V.sequence_poll() == V.VDA_OK


@pytest.mark.parametrize("room", [256, 2048])
@pytest.mark.parametrize("Hq,Hkv,d", [(2, 2, 64), (8, 2, 128)])
def test_nan_behind_the_keys_of_a_tile_with_few_rows(Hq, Hkv, d, room):
    """One query to a sequence, so three of four warps have no row; the keys end at every
    place of a block. Each zeroed row of V is one lane's."""
    lens = [room - 128 + i for i in range(1, 129)]
    N = len(lens)
    Q, K, Vv = rand(91, N, Hq, d, scale=1.5), rand(92, N * room, Hkv, d), rand(93, N * room, Hkv, d)
    for i, n in enumerate(lens):
        K[i * room + n:(i + 1) * room] = float("nan")
        Vv[i * room + n:(i + 1) * room] = float("nan")
    kr = [(i * room, i * room + n) for i, n in enumerate(lens)]
    ref = po.causal_attention(f64(Q), f64(K), f64(Vv), ranges([1] * N), kr, d ** -0.5)
    a = [t.to(DEV) for t in (Q, K, Vv)]
    kl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    first = None
    for _ in range(20):
        O = V.causal_attention(*a, starts([1] * N, DEV), cu_k=starts([room] * N, DEV), k_len=kl)
        first = O if first is None else first
        assert torch.equal(O, first)
    bounded(f64(first), ref["O"], ref["abs_O"], "O")


def _like_oracle(O, lse, ref, n):
    """Not finite exactly where the definition is not, within the bounds elsewhere."""
    o, l = f64(O)[:n], f64(lse)[:n]
    assert np.array_equal(np.isnan(o), np.isnan(ref["O"][:n]))
    assert np.array_equal(np.isnan(l), np.isnan(ref["lse"][:n]))
    bounded(o, ref["O"][:n], ref["abs_O"][:n], "O")
    assert np.array_equal(np.isneginf(l), np.isneginf(ref["lse"][:n]))


FORMS = [  # name, query and key heads, d, queries, keys to a sequence, sequences: each form that sizes choose
    ("one_stream", 1, 1, 128, 300, 300, 32),
    ("one_stream_d64", 3, 1, 64, 300, 300, 32),
    ("two_streams", 1, 1, 128, 2560, 2560, 2),
    ("few_rows", 4, 2, 128, 1, 2500, 40),
    ("few_rows_d64", 2, 2, 64, 1, 1100, 40),
    ("few_tiles", 1, 1, 128, 100, 3000, 3),
]


@pytest.mark.parametrize("kind", ["nan", "inf", "range"])
@pytest.mark.parametrize("name,Hq,Hkv,d,nq,nk,N", FORMS, ids=[f[0] for f in FORMS])
def test_logits_that_are_not_finite_are_not_hidden(name, Hq, Hkv, d, nq, nk, N, kind):
    """One key of each sequence, another place in each: NaN, infinite (so its logit is +inf for
    one query and -inf for the next), or so large that the logits leave fp32's range. A row
    that sees NaN or +inf is NaN, one that sees -inf goes without that key, one that sees
    nothing else is NaN, all others are as ever."""
    Q = rand(101, N * nq, Hq, d, scale=1.5)
    K, Vv = rand(102, N * nk, Hkv, d), rand(103, N * nk, Hkv, d)
    Q[..., 0] = torch.where(torch.arange(N * nq * Hq).view(-1, Hq) // Hq % 2 == 0, 64.0, -64.0).to(Q.dtype)
    K[..., 0] = 0.0
    for i in range(N):
        K[i * nk + (i * 3 + i // 16) % (nk - nq + 128 if nq < nk else 128), :, 0] = \
            {"nan": float("nan"), "inf": float("inf"), "range": 3e38}[kind]
    qd = f64(Q)
    with np.errstate(all="ignore"):
        kd = f64(K)
        if kind == "range":
            kd[..., 0] = np.where(kd[..., 0] > 0, np.inf, 0.0)
        ref = po.causal_attention(qd, kd, f64(Vv), ranges([nq] * N), ranges([nk] * N), d ** -0.5)
    O, lse = V.causal_attention(Q.to(DEV), K.to(DEV), Vv.to(DEV), starts([nq] * N, DEV), cu_k=starts([nk] * N, DEV),
                                return_lse=True)
    _like_oracle(O, lse, ref, N * nq)
    assert np.isnan(ref["O"]).any()


def test_a_cache_of_one_key_beyond_the_range():
    """Every logit that a row sees is -inf, in one block and in shares of several CTAs."""
    Hq, d = 2, 64
    for nk in (1, 130, 3000):
        Q = torch.full((3, Hq, d), -64.0, dtype=torch.bfloat16, device=DEV)
        K = torch.full((3 * nk, Hq, d), 3e38, dtype=torch.bfloat16, device=DEV)
        O, lse = V.causal_attention(Q, K, torch.ones_like(K), starts([1] * 3, DEV), cu_k=starts([nk] * 3, DEV),
                                    k_len=torch.tensor([nk, 0, 1], dtype=torch.int32, device=DEV), return_lse=True)
        assert torch.isnan(O[0]).all() and torch.isnan(lse[0]).all()
        assert (O[1] == 0).all() and torch.isneginf(lse[1]).all()
        assert torch.isnan(O[2]).all() and torch.isnan(lse[2]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_nan_reaches_the_gradients(d):
    """Of the sequence that has it, and of no other."""
    H, lens = 2, [200, 150, 180]
    T = sum(lens)
    Q, K, Vv, dO = (rand(111 + i, T, H, d).to(DEV) for i in range(4))
    cu = starts(lens, DEV)
    bad = 200 + 70
    K[bad, 1, 5] = float("nan")
    O, lse = V.causal_attention(Q, K, Vv, cu, return_lse=True)
    g = V.causal_attention_backward(Q, K, Vv, O, dO, lse, cu)
    assert torch.isnan(O[bad:350, 1]).all() and torch.isnan(g["dQ"][bad:350, 1]).all()
    for n in ("dK", "dV"):
        assert torch.isnan(g[n][bad, 1]).all()
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[200:350] = False
    for t in (O, *g.values()):
        assert torch.isfinite(t[:, 0]).all() and torch.isfinite(t[keep]).all()
