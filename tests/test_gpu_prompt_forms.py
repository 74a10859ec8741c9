"""The prompt path's forms that a call's sizes choose: two streams to a CTA (long
sequences at d = 128), more sequences than a warp finds by itself (33 to 128), segments
among them, and uncut sequences next to cut ones."""
import numpy as np
import pytest
import torch

from frame_level_delta_b200 import vda as V
from oracle import prompt_oracle as po
from tests.prompt_cases import bounded, f64, rand, rand32, ranges, slopes, starts

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
    assert V.sequence_poll() == 0


# name, Hq, Hkv, d, query lengths, key lengths (None: the same), spread of the logits
ATTN = [
    ("two_streams", 2, 1, 128, [2400], None, 1.5),
    ("two_streams_one_row_over", 1, 1, 128, [2561], None, 1.5),
    ("two_streams_group_3", 3, 1, 128, [2311, 2400], None, 1.5),
    ("two_streams_peaked", 1, 1, 128, [2350], None, 12.0),
    ("two_streams_long_and_short", 2, 1, 128, [5000, 1, 130], None, 1.5),
    ("two_streams_more_keys", 1, 1, 128, [1300], [2700], 1.5),
    ("two_streams_fewer_keys", 1, 1, 128, [2900], [2500], 1.5),
    ("forty_sequences", 4, 2, 128, [(i * 37) % 190 for i in range(40)], None, 1.5),
    ("hundred_sequences_d64", 2, 2, 64, [(i * 53) % 150 for i in range(100)], None, 1.5),
    ("thirty_three_group_3", 3, 1, 128, [(i * 29) % 100 for i in range(33)], None, 1.5),
]


@pytest.mark.parametrize("name,Hq,Hkv,d,nq,nk,spread", ATTN, ids=[c[0] for c in ATTN])
def test_causal_attention_forms(name, Hq, Hkv, d, nq, nk, spread):
    nk = nq if nk is None else nk
    Q = rand(3, sum(nq) + 5, Hq, d, scale=spread)
    K, Vv = rand(4, sum(nk) + 5, Hkv, d), rand(5, sum(nk) + 5, Hkv, d)
    dO = rand(9, *Q.shape)
    for t, n in ((Q, nq), (K, nk), (Vv, nk), (dO, nq)):
        t[sum(n):] = float("nan")
    ref = po.causal_attention(f64(Q), f64(K), f64(Vv), ranges(nq), ranges(nk), d ** -0.5, f64(dO))
    q, k, v, g = (t.to(DEV) for t in (Q, K, Vv, dO))
    cq, ck = starts(nq, DEV), starts(nk, DEV)
    O = torch.full_like(q, float("nan"))
    _, lse = V.causal_attention(q, k, v, cq, cu_k=ck, O=O, return_lse=True)
    bounded(f64(O), ref["O"], ref["abs_O"], "O")
    assert np.isnan(f64(O)[sum(nq):]).all()
    w, l = ref["lse"][:sum(nq)], f64(lse)[:sum(nq)]
    assert np.array_equal(np.isneginf(l), np.isneginf(w))
    ok = np.isfinite(w)
    assert np.abs(l[ok] - w[ok]).max(initial=0) <= 2.0 ** -11 + 1e-6 * np.abs(w[ok]).max(initial=0)
    out = {n: torch.full_like(t, float("nan")) for n, t in (("dQ", q), ("dK", k), ("dV", v))}
    V.causal_attention_backward(q, k, v, O, g, lse, cq, cu_k=ck, out=out)
    for n, m in (("dQ", nq), ("dK", nk), ("dV", nk)):
        bounded(f64(out[n]), ref[n], ref["abs_" + n], n)
        assert np.isnan(f64(out[n])[sum(m):]).all()


@pytest.mark.parametrize("N,room", [(40, 1100), (100, 1100)])
def test_single_tokens_of_many_caches(N, room):
    """The split form with more sequences than a warp finds by itself."""
    Hq, Hkv, d = 4, 2, 128
    lens = [(i * 277) % (room + 1) for i in range(N)]
    Q, K, Vv = rand(5, N, Hq, d, scale=1.5), rand(6, N * room, Hkv, d), rand(7, N * room, Hkv, d)
    for i, n in enumerate(lens):
        K[i * room + n:(i + 1) * room] = float("nan")
        Vv[i * room + n:(i + 1) * room] = float("nan")
    kr = [(i * room, i * room + n) for i, n in enumerate(lens)]
    ref = po.causal_attention(f64(Q), f64(K), f64(Vv), ranges([1] * N), kr, d ** -0.5)
    O = V.causal_attention(Q.to(DEV), K.to(DEV), Vv.to(DEV), starts([1] * N, DEV), cu_k=starts([room] * N, DEV),
                           k_len=torch.tensor(lens, dtype=torch.int32, device=DEV))
    bounded(f64(O), ref["O"], ref["abs_O"], "O")


DECAY = [
    ("nine_chunks_uncut", 2, 128, [1152]),
    ("ten_chunks", 2, 128, [1153]),
    ("forty_sequences_cut", 2, 64, [(i * 137) % 800 for i in range(40)]),
    ("hundred_sequences", 1, 128, [(i * 31) % 140 for i in range(100)]),
    ("thirty_two_and_a_long_one", 1, 64, [5] * 31 + [1700]),
]


@pytest.mark.parametrize("name,H,d,lens", DECAY, ids=[c[0] for c in DECAY])
def test_decay_attention_forms(name, H, d, lens):
    N, T = len(lens), sum(lens) + 4
    Q, K, Vv, dO = rand(21, T, H, d, unit=True), rand(22, T, H, d, unit=True), rand(23, T, H, d), rand(24, T, H, d)
    S0, dS = rand32(25, N, H, d, d), rand32(26, N, H, d, d)
    for t in (Q, K, Vv, dO):
        t[sum(lens):] = float("nan")
    g = slopes(H)
    ref = po.decay_attention(f64(Q), f64(K), f64(Vv), f64(g), ranges(lens), f64(S0), 0.5, f64(dO), f64(dS))
    q, k, v, do = (t.to(DEV) for t in (Q, K, Vv, dO))
    O = torch.full_like(q, float("nan"))
    _, S = V.decay_attention(q, k, v, g.to(DEV), starts(lens, DEV), S0=S0.to(DEV), scale=0.5, O=O)
    bounded(f64(O), ref["O"], ref["abs_O"], "O")
    assert np.isnan(f64(O)[sum(lens):]).all()
    r = V.decay_attention_backward(q, k, v, do, g.to(DEV), starts(lens, DEV), S0=S0.to(DEV), dS=dS.to(DEV), scale=0.5)
    for n in ("dQ", "dK", "dV"):
        bounded(f64(r[n])[:sum(lens)], ref[n][:sum(lens)], ref["abs_" + n][:sum(lens)], n)
    # fp32 states: a step rounds once (2^-24), the sums over 128 tokens in steps of 16 for
    # three parts truncate 24 times (2^-23 each)
    for got, want, s in ((S, ref["S"], ref["abs_S"]), (r["dS0"], ref["dS0"], ref["abs_dS0"])):
        assert (np.abs(f64(got) - want) <= 2.0 ** -18 * s + 1e-30).all()


def test_calls_behind_one_another_on_one_stream():
    """Calls of several launches, each of which starts under the end of the one before it:
    a call reads what the call before it wrote, and overwrites what that one read."""
    H, d, lens = 2, 64, [1700, 40, 900]
    cu, g = starts(lens, DEV), slopes(H).to(DEV)
    T = sum(lens)
    q, k, v = (rand(s, T, H, d, unit=True).to(DEV) for s in (41, 42, 43))

    def steps(sync):
        x, S = v.clone(), None
        for _ in range(6):
            x, S = V.decay_attention(q, k, x, g, cu, S0=S)
            if sync:
                torch.cuda.synchronize()
            x, lse = V.causal_attention(q, k, x, cu, return_lse=True)
            if sync:
                torch.cuda.synchronize()
            r = V.causal_attention_backward(q, k, v, x, x, lse, cu)
            x.copy_(r["dV"])
            if sync:
                torch.cuda.synchronize()
        return x, S

    a, b = steps(False), steps(True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.isfinite(a[0]).all()
