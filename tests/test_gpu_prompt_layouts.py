"""Layouts that the prompt path's calls accept beside packed ones: rows any distance apart in
either direction, heads out of a joint tensor, rooms that are filled in part, one key head for
all query heads. What lies between the rows is left as it was."""
import numpy as np
import pytest
import torch

from frame_level_delta_b200 import vda as V
from oracle import prompt_oracle as po
from tests.prompt_cases import bounded, f64, rand, rand32, ranges, slopes, starts

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MARK = 7.0


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    V.lib()


@pytest.fixture(autouse=True)
def _no_timeout():
    yield
    assert V.sequence_poll() == V.VDA_OK


def _spread(t, extra, front=8):
    """t on the device with ``extra`` elements between its token rows, ``front`` of them before
    each; everything between is MARK. Returns the view and what holds it."""
    T, H, d = t.shape
    hold = torch.full((T, H * d + extra), MARK, dtype=t.dtype, device=DEV)
    view = hold[:, front:front + H * d].view(T, H, d)
    view.copy_(t)
    return view, hold


def _untouched(hold, width, front=8):
    return bool((hold[:, :front] == MARK).all() and (hold[:, front + width:] == MARK).all())


ATTN = [
    (4, 2, 128, [150, 0, 1, 300], None),
    (6, 2, 64, [150, 1, 270], None),
    (2, 1, 128, [2400], None),              # two streams to a CTA
    (4, 1, 128, [1, 2, 1], [1500, 900, 3]),  # shares of the keys
    (3, 1, 128, [140], [400]),
]


@pytest.mark.parametrize("Hq,Hkv,d,nq,nk", ATTN)
def test_causal_attention_of_rows_apart(Hq, Hkv, d, nq, nk):
    nk = nq if nk is None else nk
    Q, dO = rand(171, sum(nq), Hq, d, scale=1.5), rand(174, sum(nq), Hq, d)
    K, Vv = rand(172, sum(nk), Hkv, d), rand(173, sum(nk), Hkv, d)
    ref = po.causal_attention(f64(Q), f64(K), f64(Vv), ranges(nq), ranges(nk), d ** -0.5, f64(dO))
    cq, ck = starts(nq, DEV), starts(nk, DEV)
    q, _ = _spread(Q, 24)
    k, _ = _spread(K, 8)
    v, _ = _spread(Vv, 136)
    O, hold = _spread(torch.zeros_like(Q), 40)
    _, lse = V.causal_attention(q, k, v, cq, cu_k=ck, O=O, return_lse=True)
    bounded(f64(O), ref["O"], ref["abs_O"], "O")
    assert _untouched(hold, Hq * d)
    g, _ = _spread(dO, 40)
    r = V.causal_attention_backward(q, k, v, O, g, lse, cq, cu_k=ck)
    for n in ("dQ", "dK", "dV"):
        assert r[n].is_contiguous()
        bounded(f64(r[n]), ref[n], ref["abs_" + n], n)
    # and the same bits as packed rows give
    a = [t.contiguous() for t in (q, k, v)]
    O2, lse2 = V.causal_attention(*a, cq, cu_k=ck, return_lse=True)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    r2 = V.causal_attention_backward(*a, O2, dO.to(DEV), lse2, cq, cu_k=ck)
    assert all(torch.equal(r[n], r2[n]) for n in r)


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (3, 3, 64)])
def test_gradients_of_rooms_filled_in_part(Hq, Hkv, d):
    """k_len: keys behind the filled part hold NaN, give nothing and keep their gradients' rows."""
    nq, room, fill = [130, 1, 40, 5], [300, 200, 40, 130], [257, 0, 17, 129]
    Q, dO = rand(181, sum(nq), Hq, d, scale=1.5), rand(184, sum(nq), Hq, d)
    K, Vv = rand(182, sum(room), Hkv, d), rand(183, sum(room), Hkv, d)
    kr = [(a, a + n) for (a, _), n in zip(ranges(room), fill)]
    behind = torch.ones(sum(room), dtype=torch.bool)
    for a, b in kr:
        behind[a:b] = False
    K[behind], Vv[behind] = float("nan"), float("nan")
    ref = po.causal_attention(f64(Q), f64(K), f64(Vv), ranges(nq), kr, d ** -0.5, f64(dO))
    q, k, v, g = (t.to(DEV) for t in (Q, K, Vv, dO))
    at = dict(cu_k=starts(room, DEV), k_len=torch.tensor(fill, dtype=torch.int32, device=DEV))
    O, lse = V.causal_attention(q, k, v, starts(nq, DEV), return_lse=True, **at)
    bounded(f64(O), ref["O"], ref["abs_O"], "O")
    out = {n: torch.full_like(t, MARK) for n, t in (("dQ", q), ("dK", k), ("dV", v))}
    V.causal_attention_backward(q, k, v, O, g, lse, starts(nq, DEV), out=out, **at)
    bounded(f64(out["dQ"]), ref["dQ"], ref["abs_dQ"], "dQ")
    for n in ("dK", "dV"):
        bounded(f64(out[n])[~behind.numpy()], ref[n][~behind.numpy()], ref["abs_" + n][~behind.numpy()], n)
        assert (out[n][behind.to(DEV)] == MARK).all(), n
    # a length beyond the room is held to it, one below 0 is none
    full = V.causal_attention(q, k, v, starts(nq, DEV), cu_k=at["cu_k"],
                              k_len=torch.tensor([257, -3, 17, 129], dtype=torch.int32, device=DEV))
    assert torch.equal(full, O)


@pytest.mark.parametrize("Hq,d", [(128, 64), (127, 64), (65, 128), (96, 128)])
def test_many_query_heads_to_one_key_head(Hq, d):
    """One token to a tile, so each row of a tile is another head (not always 128 of them)."""
    nq, nk = [3, 40, 1], [3, 70, 130]
    Q, dO = rand(191, sum(nq), Hq, d, scale=1.5), rand(194, sum(nq), Hq, d)
    K, Vv = rand(192, sum(nk), 1, d), rand(193, sum(nk), 1, d)
    ref = po.causal_attention(f64(Q), f64(K), f64(Vv), ranges(nq), ranges(nk), d ** -0.5, f64(dO))
    q, k, v, g = (t.to(DEV) for t in (Q, K, Vv, dO))
    at = dict(cu_k=starts(nk, DEV))
    O, lse = V.causal_attention(q, k, v, starts(nq, DEV), return_lse=True, **at)
    bounded(f64(O), ref["O"], ref["abs_O"], "O")
    r = V.causal_attention_backward(q, k, v, O, g, lse, starts(nq, DEV), **at)
    for n in ("dQ", "dK", "dV"):
        bounded(f64(r[n]), ref[n], ref["abs_" + n], n)


@pytest.mark.parametrize("H,d,lens", [(3, 128, [300, 0, 1, 128]), (2, 64, [257, 128, 5]), (2, 128, [1500, 40])])
def test_decay_attention_of_rows_apart(H, d, lens):
    T, N = sum(lens), len(lens)
    Q, K, Vv, dO = rand(201, T, H, d, unit=True), rand(202, T, H, d, unit=True), rand(203, T, H, d), rand(204, T, H, d)
    S0, dS, ld = rand32(205, N, H, d, d), rand32(206, N, H, d, d), slopes(H)
    ref = po.decay_attention(f64(Q), f64(K), f64(Vv), f64(ld), ranges(lens), f64(S0), 0.5, f64(dO), f64(dS))
    g, cu, s0, ds = ld.to(DEV), starts(lens, DEV), S0.to(DEV), dS.to(DEV)
    q, _ = _spread(Q, 24)
    k, _ = _spread(K, 8)
    v, _ = _spread(Vv, 136)
    up, _ = _spread(dO, 16)
    O, hold = _spread(torch.zeros_like(Q), 40)
    _, S = V.decay_attention(q, k, v, g, cu, S0=s0, scale=0.5, O=O)
    bounded(f64(O), ref["O"], ref["abs_O"], "O")
    assert _untouched(hold, H * d)
    a = [t.contiguous() for t in (q, k, v)]
    O2, S2 = V.decay_attention(*a, g, cu, S0=s0, scale=0.5)
    assert torch.equal(O, O2) and torch.equal(S, S2)
    r = V.decay_attention_backward(q, k, v, up, g, cu, S0=s0, dS=ds, scale=0.5)
    r2 = V.decay_attention_backward(*a, dO.to(DEV), g, cu, S0=s0, dS=ds, scale=0.5)
    for n in r:
        assert torch.equal(r[n], r2[n]), n
    for n in ("dQ", "dK", "dV"):
        bounded(f64(r[n]), ref[n], ref["abs_" + n], n)


@pytest.mark.parametrize("N,H,d", [(5, 3, 128), (200, 4, 64)])
def test_step_of_rows_apart(N, H, d):
    Q, K, Vv = rand(211, N, H, d, unit=True), rand(212, N, H, d, unit=True), rand(213, N, H, d)
    S0, g = rand32(214, N, H, d, d), slopes(H).to(DEV)
    S, S2 = S0.to(DEV), S0.to(DEV)
    q, _ = _spread(Q, 24)
    k, _ = _spread(K, 8)
    v, _ = _spread(Vv, 136)
    O, hold = _spread(torch.zeros_like(Q), 40)
    V.decay_attention_step(q, k, v, g, S, O=O)
    assert _untouched(hold, H * d)
    O2 = V.decay_attention_step(Q.to(DEV), K.to(DEV), Vv.to(DEV), g, S2)
    assert torch.equal(O, O2) and torch.equal(S, S2)


def test_one_token_at_any_distance():
    """Of a tensor of one row the distance to the next is never used."""
    H, d = 2, 64
    x = rand(221, 1, H, d, unit=True).to(DEV)
    odd = x.as_strided((1, H, d), (3, d, 1))
    cu, g = starts([1], DEV), slopes(H).to(DEV)
    assert torch.equal(V.causal_attention(odd, odd, odd, cu), V.causal_attention(x, x, x, cu))
    assert torch.equal(V.decay_attention(odd, odd, odd, g, cu)[0], V.decay_attention(x, x, x, g, cu)[0])
