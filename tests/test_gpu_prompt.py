"""The prompt path on the GPU against the float64 oracle: causal attention over packed
sequences (forward, single tokens, gradients) and decayed linear attention (prompts,
single tokens, gradients)."""
import numpy as np
import pytest
import torch

from frame_level_delta_b200 import vda as V
from oracle import prompt_oracle as po
from tests.prompt_cases import U, bounded, f64, rand, rand32, ranges, slopes, starts

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


# ------------------------------------------------------------------ causal attention
# name, Hq, Hkv, d, query lengths, key lengths (None: the same), spread of the logits
ATTN = [
    ("one_token", 2, 2, 128, [1], None, 1.0),
    ("one_tile", 2, 1, 128, [128], None, 1.0),
    ("two_tiles_edge", 1, 1, 128, [129], None, 1.0),
    ("ragged", 4, 2, 128, [1, 127, 0, 128, 129, 300, 2], None, 1.5),
    ("ragged_d64", 4, 2, 64, [5, 257, 0, 64, 1], None, 1.5),
    ("group_3", 6, 2, 128, [130, 45, 300], None, 1.5),
    ("group_5_d64", 5, 1, 64, [77, 200], None, 1.5),
    ("group_128", 128, 1, 64, [3, 40], None, 1.0),
    ("peaked", 2, 2, 128, [400, 33], None, 12.0),
    ("more_keys", 4, 2, 128, [3, 130, 60], [200, 140, 60], 1.5),
    ("fewer_keys", 4, 2, 128, [200, 10, 140], [150, 0, 13], 1.5),
    ("many_sequences", 2, 1, 64, [i % 4 for i in range(700)], None, 1.0),
    ("long", 2, 1, 128, [1200], None, 1.5),
    ("long_few_rows", 4, 2, 128, [7], [2500], 1.5),
    ("chunk_on_cache", 8, 2, 64, [40, 9, 1], [3000, 1, 1300], 1.5),
]


def _attn_inputs(Hq, Hkv, d, nq, nk, spread, seed=3, tail=5):
    nk = nq if nk is None else nk
    Tq, Tk = sum(nq) + tail, sum(nk) + tail
    Q = rand(seed, Tq, Hq, d, scale=spread)
    K, Vv = rand(seed + 1, Tk, Hkv, d), rand(seed + 2, Tk, Hkv, d)
    # What lies behind the last sequence must not matter.
    for t, n in ((Q, nq), (K, nk), (Vv, nk)):
        t[sum(n):] = float("nan")
        t[sum(n) + 1:] = float("inf")
    return Q, K, Vv, nk


def _check_attn(O, lse, ref, n):
    bounded(f64(O), ref["O"], ref["abs_O"], "O")
    assert np.isnan(f64(O)[n:]).all()  # rows behind the last sequence are left as they were
    w = ref["lse"][:n]
    g = f64(lse)[:n]
    assert np.array_equal(np.isneginf(g), np.isneginf(w))
    ok = np.isfinite(w)
    assert np.abs(g[ok] - w[ok]).max(initial=0) <= 2.0 ** -11 + 1e-6 * np.abs(w[ok]).max(initial=0)


@pytest.mark.parametrize("name,Hq,Hkv,d,nq,nk,spread", ATTN, ids=[c[0] for c in ATTN])
def test_causal_attention(name, Hq, Hkv, d, nq, nk, spread):
    Q, K, Vv, nk = _attn_inputs(Hq, Hkv, d, nq, nk, spread)
    ref = po.causal_attention(f64(Q), f64(K), f64(Vv), ranges(nq), ranges(nk), d ** -0.5)
    O = torch.full_like(Q, float("nan"), device=DEV)
    _, lse = V.causal_attention(Q.to(DEV), K.to(DEV), Vv.to(DEV), starts(nq, DEV), cu_k=starts(nk, DEV), O=O,
                                return_lse=True)
    _check_attn(O, lse, ref, sum(nq))


def test_causal_attention_without_keys_or_tokens():
    Q, K, Vv = rand(0, 9, 2, 64).to(DEV), rand(1, 0, 2, 64).to(DEV), rand(2, 0, 2, 64).to(DEV)
    O, lse = V.causal_attention(Q, K, Vv, starts([4, 5], DEV), cu_k=starts([0, 0], DEV), return_lse=True)
    assert (O == 0).all() and torch.isneginf(lse).all()
    e = Q[:0]
    assert V.causal_attention(e, e, e, starts([0], DEV)).shape == (0, 2, 64)


@pytest.mark.parametrize("Hq,Hkv,d,room,lens", [
    (8, 8, 128, 300, [1, 300, 128, 129, 0, 57]),
    (8, 2, 128, 2048, [2048, 1, 1000, 129, 0]),
    (24, 8, 128, 4096, [4095, 3]),
    (7, 1, 64, 1500, [1500, 700, 12]),
    (2, 1, 64, 40000, [40000]),
])
def test_single_tokens_against_a_cache(Hq, Hkv, d, room, lens):
    """One query per sequence; a cache's unfilled room holds NaN."""
    N = len(lens)
    Q, K, Vv = rand(5, N, Hq, d, scale=1.5), rand(6, N * room, Hkv, d), rand(7, N * room, Hkv, d)
    for i, n in enumerate(lens):
        K[i * room + n:(i + 1) * room] = float("nan")
        Vv[i * room + n:(i + 1) * room] = float("nan")
    kr = [(i * room, i * room + n) for i, n in enumerate(lens)]
    ref = po.causal_attention(f64(Q), f64(K), f64(Vv), ranges([1] * N), kr, d ** -0.5)
    O, lse = V.causal_attention(Q.to(DEV), K.to(DEV), Vv.to(DEV), starts([1] * N, DEV),
                                cu_k=starts([room] * N, DEV), k_len=torch.tensor(lens, dtype=torch.int32, device=DEV),
                                return_lse=True)
    bounded(f64(O), ref["O"], ref["abs_O"], "O")
    w, g = ref["lse"], f64(lse)
    assert np.array_equal(np.isneginf(g), np.isneginf(w))
    ok = np.isfinite(w)
    assert np.abs(g[ok] - w[ok]).max() <= 2.0 ** -11


def test_causal_attention_of_a_joint_projection_and_of_head_slices():
    """Q, K, V as parts of one [tokens, (Hq + 2 Hkv) d] tensor, and a slice of the heads."""
    Hq, Hkv, d, lens = 4, 2, 128, [150, 70]
    T = sum(lens)
    joint = rand(11, T, Hq + 2 * Hkv, d).to(DEV)
    Q, K, Vv = joint[:, :Hq], joint[:, Hq:Hq + Hkv], joint[:, Hq + Hkv:]
    cu = starts(lens, DEV)
    want = V.causal_attention(Q.contiguous(), K.contiguous(), Vv.contiguous(), cu)
    assert torch.equal(V.causal_attention(Q, K, Vv, cu), want)
    O = torch.full_like(Q.contiguous(), 7.0)
    V.causal_attention(Q[:, 2:], K[:, 1:], Vv[:, 1:], cu, O=O[:, 2:])
    assert torch.equal(O[:, 2:], want[:, 2:]) and (O[:, :2] == 7).all()


BWD = [c for c in ATTN if c[0] not in ("group_128", "many_sequences")] + [
    ("many_short", 2, 1, 64, [i % 3 for i in range(400)], None, 1.0)]


@pytest.mark.parametrize("name,Hq,Hkv,d,nq,nk,spread", BWD, ids=[c[0] for c in BWD])
def test_causal_attention_backward(name, Hq, Hkv, d, nq, nk, spread):
    Q, K, Vv, nk = _attn_inputs(Hq, Hkv, d, nq, nk, spread)
    dO = rand(9, *Q.shape)
    dO[sum(nq):] = float("nan")
    ref = po.causal_attention(f64(Q), f64(K), f64(Vv), ranges(nq), ranges(nk), d ** -0.5, f64(dO))
    cq, ck = starts(nq, DEV), starts(nk, DEV)
    q, k, v, g = (t.to(DEV) for t in (Q, K, Vv, dO))
    O, lse = V.causal_attention(q, k, v, cq, cu_k=ck, return_lse=True)
    out = {n: torch.full_like(t, float("nan")) for n, t in (("dQ", q), ("dK", k), ("dV", v))}
    V.causal_attention_backward(q, k, v, O, g, lse, cq, cu_k=ck, out=out)
    for n, m in (("dQ", nq), ("dK", nk), ("dV", nk)):
        bounded(f64(out[n]), ref[n], ref["abs_" + n], n)
        assert np.isnan(f64(out[n])[sum(m):]).all()
    again = V.causal_attention_backward(q, k, v, O, g, lse, cq, cu_k=ck)
    for n, m in (("dQ", nq), ("dK", nk), ("dV", nk)):
        assert torch.equal(again[n][:sum(m)], out[n][:sum(m)])


# ------------------------------------------------------------------ decayed linear attention
DECAY = [
    ("one_token", 2, 128, [1], 1.0),
    ("one_chunk", 2, 128, [128], 1.0),
    ("ragged", 3, 128, [1, 127, 0, 128, 129, 300, 2], 1.0),
    ("ragged_d64", 3, 64, [5, 257, 0, 64, 1], 0.25),
    ("segments", 2, 128, [2500], 1.0),
    ("segments_ragged", 2, 64, [1100, 3, 1025, 0, 2049], 1.0),
    ("many_sequences", 1, 64, [i % 3 for i in range(500)], 1.0),
]


def _decay_inputs(H, d, lens, seed=21, tail=4):
    T = sum(lens) + tail
    Q, K, Vv = rand(seed, T, H, d, unit=True), rand(seed + 1, T, H, d, unit=True), rand(seed + 2, T, H, d)
    dO = rand(seed + 3, T, H, d)
    for t in (Q, K, Vv, dO):
        t[sum(lens):] = float("nan")
    return Q, K, Vv, dO, rand32(seed + 4, len(lens), H, d, d), rand32(seed + 5, len(lens), H, d, d)


def _check_state(got, want, abs_sum):
    """fp32 states: three bf16 parts of an operand hold 24 bits, a step of the
    recurrence rounds once (2^-24), and the tensor cores' sums over 128 tokens in
    steps of 16 for three parts truncate 24 times (2^-23 each)."""
    tol = 2.0 ** -18 * abs_sum + 1e-30
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol)
    assert np.linalg.norm(got - want) <= 4e-6 * np.linalg.norm(want)


@pytest.mark.parametrize("state", [True, False], ids=["state", "zero"])
@pytest.mark.parametrize("name,H,d,lens,scale", DECAY, ids=[c[0] for c in DECAY])
def test_decay_attention(name, H, d, lens, scale, state):
    Q, K, Vv, _, S0, _ = _decay_inputs(H, d, lens)
    g = slopes(H)
    if not state:
        S0 = torch.zeros_like(S0)
    ref = po.decay_attention(f64(Q), f64(K), f64(Vv), f64(g), ranges(lens), f64(S0), scale)
    O = torch.full_like(Q, float("nan"), device=DEV)
    s0 = S0.to(DEV) if state else None
    _, S = V.decay_attention(Q.to(DEV), K.to(DEV), Vv.to(DEV), g.to(DEV), starts(lens, DEV), S0=s0, scale=scale, O=O)
    bounded(f64(O), ref["O"], ref["abs_O"], "O")
    assert np.isnan(f64(O)[sum(lens):]).all()
    _check_state(f64(S), ref["S"], ref["abs_S"])
    if state:  # the state updated in place
        V.decay_attention(Q.to(DEV), K.to(DEV), Vv.to(DEV), g.to(DEV), starts(lens, DEV), S0=s0, S=s0, scale=scale)
        assert torch.equal(s0, S)


@pytest.mark.parametrize("g", [0.0, -1e-4, -0.7, -30.0, -1e4, float("-inf")])
def test_decay_attention_decays(g):
    """From a head that keeps everything to one that keeps nothing."""
    H, d, lens = 2, 64, [200, 77]
    Q, K, Vv, dO, S0, dS = _decay_inputs(H, d, lens)
    ld = torch.full((H,), g)
    with np.errstate(over="ignore"):
        ref = po.decay_attention(f64(Q), f64(K), f64(Vv), f64(ld), ranges(lens), f64(S0), 1.0, f64(dO), f64(dS))
    a = [t.to(DEV) for t in (Q, K, Vv)]
    O, S = V.decay_attention(*a, ld.to(DEV), starts(lens, DEV), S0=S0.to(DEV))
    bounded(f64(O), ref["O"], ref["abs_O"], "O")
    _check_state(f64(S), ref["S"], ref["abs_S"])
    r = V.decay_attention_backward(*a, dO.to(DEV), ld.to(DEV), starts(lens, DEV), S0=S0.to(DEV), dS=dS.to(DEV))
    for n in ("dQ", "dK", "dV"):
        bounded(f64(r[n]), ref[n], ref["abs_" + n], n)
    _check_state(f64(r["dS0"]), ref["dS0"], ref["abs_dS0"])


@pytest.mark.parametrize("name,H,d,lens,scale", DECAY, ids=[c[0] for c in DECAY])
def test_decay_attention_backward(name, H, d, lens, scale):
    Q, K, Vv, dO, S0, dS = _decay_inputs(H, d, lens)
    g = slopes(H)
    ref = po.decay_attention(f64(Q), f64(K), f64(Vv), f64(g), ranges(lens), f64(S0), scale, f64(dO), f64(dS))
    q, k, v, do = (t.to(DEV) for t in (Q, K, Vv, dO))
    out = {n: torch.full_like(q, float("nan")) for n in ("dQ", "dK", "dV")}
    out["dS0"] = torch.full_like(S0, float("nan"), device=DEV)
    V.decay_attention_backward(q, k, v, do, g.to(DEV), starts(lens, DEV), S0=S0.to(DEV), dS=dS.to(DEV), scale=scale,
                               out=out)
    for n in ("dQ", "dK", "dV"):
        bounded(f64(out[n]), ref[n], ref["abs_" + n], n)
        assert np.isnan(f64(out[n])[sum(lens):]).all()
    _check_state(f64(out["dS0"]), ref["dS0"], ref["abs_dS0"])


def test_decay_attention_backward_without_states():
    """No initial state, no gradient of the last one, dS0 not wanted."""
    H, d, lens = 2, 128, [200, 0, 1400]
    Q, K, Vv, dO, S0, _ = _decay_inputs(H, d, lens)
    g, zero = slopes(H), np.zeros(S0.shape)
    ref = po.decay_attention(f64(Q), f64(K), f64(Vv), f64(g), ranges(lens), zero, 1.0, f64(dO), zero)
    q, k, v, do = (t.to(DEV) for t in (Q, K, Vv, dO))
    out = {n: torch.full_like(q, float("nan")) for n in ("dQ", "dK", "dV")}
    V.decay_attention_backward(q, k, v, do, g.to(DEV), starts(lens, DEV), out=out)
    for n in ("dQ", "dK", "dV"):
        bounded(f64(out[n]), ref[n], ref["abs_" + n], n)


def test_nothing_to_do():
    """No tokens on one side or on both: gradients of unseen keys are 0, states stay."""
    H, d = 2, 64
    x = rand(1, 6, H, d).to(DEV)
    e = x[:0]
    none, six = starts([0], DEV), starts([6], DEV)
    f = dict(device=DEV, dtype=torch.float32)
    r = V.causal_attention_backward(e, x, x, e, e, torch.empty(0, H, **f), none, cu_k=six)
    assert (r["dK"] == 0).all() and (r["dV"] == 0).all() and r["dQ"].shape == e.shape
    O, lse = V.causal_attention(x, e, e, six, cu_k=none, return_lse=True)
    r = V.causal_attention_backward(x, e, e, O, x, lse, six, cu_k=none)
    assert (r["dQ"] == 0).all()
    g, S0 = slopes(H).to(DEV), rand32(3, 1, H, d, d).to(DEV)
    O, S = V.decay_attention(e, e, e, g, none, S0=S0)
    assert torch.equal(S, S0) and O.shape == e.shape
    _, S = V.decay_attention(e, e, e, g, none)
    assert (S == 0).all()
    r = V.decay_attention_backward(e, e, e, e, g, none, dS=S0)
    assert torch.equal(r["dS0"], S0)
    assert V.decay_attention_step(e, e, e, g, S0[:0]).shape == e.shape


@pytest.mark.parametrize("N,H,d", [(1, 1, 128), (1, 24, 128), (3, 5, 64), (70, 8, 128), (300, 2, 64)])
def test_decay_step(N, H, d):
    Q, K, Vv = rand(31, N, H, d, unit=True), rand(32, N, H, d, unit=True), rand(33, N, H, d)
    S0, g = rand32(34, N, H, d, d), slopes(H)
    S = S0.to(DEV)
    O = V.decay_attention_step(Q.to(DEV), K.to(DEV), Vv.to(DEV), g.to(DEV), S, scale=0.5)
    ref = po.decay_attention(f64(Q), f64(K), f64(Vv), f64(g), ranges([1] * N), f64(S0), 0.5)
    # fp32 throughout; the output is rounded once, sums of 128 terms are off by 2^-17 of their absolute values at most
    tol = U * np.abs(ref["O"]) + 2.0 ** -16 * ref["abs_O"]
    assert (np.abs(f64(O) - ref["O"]) <= tol).all()
    assert (np.abs(f64(S) - ref["S"]) <= 2.0 ** -21 * ref["abs_S"]).all()
