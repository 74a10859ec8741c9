"""The prompt path's results next to 64 bits in the 2-norm: no further off than the roundings
that the kernels make (prompt_norms.py), at lengths where outputs are far smaller than the
values they are made of."""
import numpy as np
import pytest
import torch

from frame_level_delta_b200 import vda as V
from oracle import prompt_oracle as po
from tests import prompt_norms as pn
from tests.prompt_cases import f64, rand, rand32, ranges, slopes, starts

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


def _near(got, want, abs_sum, squares, terms, what):
    live = ~np.isnan(want)
    g, w = got[live], want[live]
    lim = pn.limit(squares[live], w, abs_sum[live], terms)
    err = pn.off(g, w)
    print(f"{what}: {err / np.linalg.norm(w):.2e} of the norm, {err / lim:.2f} of the limit")
    assert err <= lim, f"{what}: {err / lim:.2f} of the limit"


# name, Hq, Hkv, d, query lengths, key lengths (None: the same), spread of the logits
ATTN = [
    ("one_tile", 4, 4, 128, [128], None, 1.0),
    ("ragged", 4, 2, 128, [1, 127, 0, 128, 129, 300, 2], None, 1.5),
    ("ragged_d64", 4, 2, 64, [5, 257, 0, 64, 300], None, 1.5),
    ("group_3", 6, 2, 128, [130, 45, 300], None, 1.5),
    ("peaked", 2, 2, 128, [400, 33], None, 12.0),
    ("more_keys", 4, 2, 128, [3, 130, 60], [200, 140, 60], 1.5),
    ("long", 2, 1, 128, [1200], None, 1.5),
    ("flat", 2, 2, 64, [1500], None, 0.1),
    ("two_streams", 2, 1, 128, [2400], None, 1.5),
    ("chunk_on_cache", 8, 2, 64, [40, 9, 1], [3000, 1, 1300], 1.5),
    ("few_tiles", 4, 1, 128, [100], [3000], 1.5),
]


@pytest.mark.parametrize("name,Hq,Hkv,d,nq,nk,spread", ATTN, ids=[c[0] for c in ATTN])
def test_causal_attention(name, Hq, Hkv, d, nq, nk, spread):
    nk = nq if nk is None else nk
    Q, dO = rand(151, sum(nq), Hq, d, scale=spread), rand(154, sum(nq), Hq, d)
    K, Vv = rand(152, sum(nk), Hkv, d), rand(153, sum(nk), Hkv, d)
    a = (*(f64(t) for t in (Q, K, Vv)), ranges(nq), ranges(nk), d ** -0.5, f64(dO))
    ref, sq = po.causal_attention(*a), pn.attention(*a)
    q, k, v, g = (t.to(DEV) for t in (Q, K, Vv, dO))
    cq, ck = starts(nq, DEV), starts(nk, DEV)
    O, lse = V.causal_attention(q, k, v, cq, cu_k=ck, return_lse=True)
    r = V.causal_attention_backward(q, k, v, O, g, lse, cq, cu_k=ck)
    for n, x in (("O", O), ("dQ", r["dQ"]), ("dK", r["dK"]), ("dV", r["dV"])):
        _near(f64(x), ref[n], ref["abs_" + n], sq[n], max(nk) if n in ("O", "dQ") else Hq // Hkv * max(nq), n)


@pytest.mark.parametrize("Hq,Hkv,d,room,lens", [
    (8, 2, 128, 2048, [2048, 1, 1000, 129]),
    (24, 8, 128, 4096, [4095, 3]),
    (8, 1, 64, 40000, [40000]),
    (16, 4, 64, 1100, [1100 - 9 * i for i in range(40)]),
])
def test_single_tokens_on_caches(Hq, Hkv, d, room, lens):
    N = len(lens)
    Q, K, Vv = rand(155, N, Hq, d, scale=1.5), rand(156, N * room, Hkv, d), rand(157, N * room, Hkv, d)
    a = (*(f64(t) for t in (Q, K, Vv)), ranges([1] * N), [(i * room, i * room + n) for i, n in enumerate(lens)], d ** -0.5)
    ref, sq = po.causal_attention(*a), pn.attention(*a)
    O = V.causal_attention(Q.to(DEV), K.to(DEV), Vv.to(DEV), starts([1] * N, DEV), cu_k=starts([room] * N, DEV),
                           k_len=torch.tensor(lens, dtype=torch.int32, device=DEV))
    _near(f64(O), ref["O"], ref["abs_O"], sq["O"], max(lens), "O")


DECAY = [
    ("ragged", 3, 128, [1, 127, 0, 128, 129, 300, 2]),
    ("ragged_d64", 3, 64, [5, 257, 0, 64, 300]),
    ("segments", 2, 128, [1500]),
    ("segments_ragged", 2, 64, [1100, 3, 1025]),
]


@pytest.mark.parametrize("name,H,d,lens", DECAY, ids=[c[0] for c in DECAY])
def test_decay_attention(name, H, d, lens):
    T, N = sum(lens), len(lens)
    Q, K, Vv, dO = rand(161, T, H, d, unit=True), rand(162, T, H, d, unit=True), rand(163, T, H, d), rand(164, T, H, d)
    S0, dS, g = rand32(165, N, H, d, d), rand32(166, N, H, d, d), slopes(H)
    a = (*(f64(t) for t in (Q, K, Vv, g)), ranges(lens), f64(S0), 0.5, f64(dO), f64(dS))
    ref, sq = po.decay_attention(*a), pn.decay(*a)
    q, k, v, do = (t.to(DEV) for t in (Q, K, Vv, dO))
    cu = starts(lens, DEV)
    O, _ = V.decay_attention(q, k, v, g.to(DEV), cu, S0=S0.to(DEV), scale=0.5)
    r = V.decay_attention_backward(q, k, v, do, g.to(DEV), cu, S0=S0.to(DEV), dS=dS.to(DEV), scale=0.5)
    for n, x in (("O", O), ("dQ", r["dQ"]), ("dK", r["dK"]), ("dV", r["dV"])):
        _near(f64(x), ref[n], ref["abs_" + n], sq[n], 2 * 128, n)
