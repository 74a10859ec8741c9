"""The prompt path as a program uses it: both operators of a hybrid layer on the same
packed prompts and their merge, prompts followed by single tokens, captured and replayed
calls, other streams, wrong prefix arrays, refusals."""
import numpy as np
import pytest
import torch

from frame_level_delta_b200 import vda as V
from oracle import prompt_oracle as po
from tests.prompt_cases import FP32, U, bounded, f64, rand, rand32, ranges, slopes, starts

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


def _case(seed, lens, Hq, Hkv, d):
    T = sum(lens)
    t = [rand(seed, T, Hq, d, unit=True, scale=1.0), rand(seed + 1, T, Hkv, d, unit=True), rand(seed + 2, T, Hkv, d)]
    return [x.to(DEV) for x in t], starts(lens, DEV)


def test_hybrid_layer_on_packed_prompts():
    """Softmax and decayed linear attention on the same tokens, merged by their output
    projections: the framework's merge takes what both return."""
    lens, H, d, N = [70, 1, 200], 4, 64, 96
    (Q, K, Vv), cu = _case(1, lens, H, H, d)
    g = slopes(H).to(DEV)
    Ws, Wl = rand(8, N, H * d, scale=(H * d) ** -0.5).to(DEV), rand(9, N, H * d, scale=(H * d) ** -0.5).to(DEV)
    Os = V.causal_attention(Q, K, Vv, cu, scale=4.0)
    Ol, _ = V.decay_attention(Q, K, Vv, g, cu)
    Y = V.hybrid_merge(Os.flatten(1), Ws, Ol.flatten(1), Wl)
    q, k, v = f64(Q), f64(K), f64(Vv)
    rs = po.causal_attention(q, k, v, ranges(lens), ranges(lens), 4.0)
    rl = po.decay_attention(q, k, v, f64(g), ranges(lens), np.zeros((len(lens), H, d, d)), 1.0)
    T = sum(lens)
    want = rs["O"].reshape(T, -1) @ f64(Ws).T + rl["O"].reshape(T, -1) @ f64(Wl).T
    # The two inputs of the merge are off by their own bounds, its output is rounded once.
    off = [((U + FP32) * r["abs_O"] + U * np.abs(r["O"])).reshape(T, -1) for r in (rs, rl)]
    tol = 1.01 * (off[0] @ np.abs(f64(Ws)).T + off[1] @ np.abs(f64(Wl)).T + U * np.abs(want)) + FP32
    assert (np.abs(f64(Y) - want) <= tol).all()


def test_prompt_then_single_tokens():
    """A prompt and then token by token gives what the whole sequence gives at once."""
    lens, more, Hq, Hkv, d, room = [33, 128, 200], 3, 4, 2, 128, 256
    N, whole = len(lens), [n + more for n in lens]
    (Q, K, Vv), cu = _case(5, whole, Hq, Hkv, d)
    g = slopes(Hkv).to(DEV)
    want = V.causal_attention(Q, K, Vv, cu, scale=3.0)
    want_l, want_S = V.decay_attention(Q[:, :Hkv], K, Vv, g, cu)
    at = [a for a, _ in ranges(whole)]
    # the prompts
    keep = torch.cat([torch.arange(a, a + n) for a, n in zip(at, lens)]).to(DEV)
    cp = starts(lens, DEV)
    got = V.causal_attention(Q[keep], K[keep], Vv[keep], cp, scale=3.0)
    got_l, S = V.decay_attention(Q[keep][:, :Hkv], K[keep], Vv[keep], g, cp)
    assert torch.equal(got, want[keep])
    kc = torch.full((N * room, Hkv, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    vc = kc.clone()
    for i, (a, n) in enumerate(zip(at, lens)):
        kc[i * room:i * room + n], vc[i * room:i * room + n] = K[a:a + n], Vv[a:a + n]
    rooms, ones = starts([room] * N, DEV), starts([1] * N, DEV)
    for t in range(more):
        rows = torch.tensor([a + n + t for a, n in zip(at, lens)], device=DEV)
        slot = torch.tensor([i * room + n + t for i, n in enumerate(lens)], device=DEV)
        kc[slot], vc[slot] = K[rows], Vv[rows]
        k_len = torch.tensor([n + t + 1 for n in lens], dtype=torch.int32, device=DEV)
        o = V.causal_attention(Q[rows], kc, vc, ones, cu_k=rooms, k_len=k_len, scale=3.0)
        # Same formula, other order of blocks: both are off by the bound of the tests at most.
        v = 1.01 * (2 * (U + FP32) * f64(Vv).max() + 2 * U * np.abs(f64(want[rows])))
        assert (np.abs(f64(o) - f64(want[rows])) <= v).all()
        ol = V.decay_attention_step(Q[rows][:, :Hkv].contiguous(), K[rows], Vv[rows], g, S)
        ref = f64(want_l[rows])
        assert np.linalg.norm(f64(ol) - ref) <= 3 * U * np.linalg.norm(ref)
    assert np.linalg.norm(f64(S) - f64(want_S)) <= 4e-6 * np.linalg.norm(f64(want_S))


def _everything(Q, K, Vv, dO, cu, g, S0, dS):
    O, lse = V.causal_attention(Q, K, Vv, cu, return_lse=True)
    r = V.causal_attention_backward(Q, K, Vv, O, dO, lse, cu)
    D, S = V.decay_attention(Q, K, Vv, g, cu, S0=S0)
    b = V.decay_attention_backward(Q, K, Vv, dO, g, cu, S0=S0, dS=dS)
    X = S.clone()
    N = S.shape[0]
    s = V.decay_attention_step(Q[:N], K[:N], Vv[:N], g, X)
    one = V.causal_attention(Q[:N], K, Vv, torch.arange(N + 1, dtype=torch.int32, device=Q.device), cu_k=cu)
    return [O, lse, *r.values(), D, S, *b.values(), X, s, one]


def _all_inputs(seed, lens, H, d):
    T, N = sum(lens), len(lens)
    Q, K, Vv, dO = (rand(seed + i, T, H, d, unit=i < 2).to(DEV) for i in range(4))
    return Q, K, Vv, dO, starts(lens, DEV), slopes(H).to(DEV), rand32(seed + 5, N, H, d, d).to(DEV), \
        rand32(seed + 6, N, H, d, d).to(DEV)


@pytest.mark.parametrize("lens,H,d", [([300, 1, 128], 3, 128), ([2500, 40], 2, 64)])
def test_captured_and_replayed(lens, H, d):
    """Two graphs of the same calls, replayed with new inputs in turn."""
    a, b = _all_inputs(40, lens, H, d), _all_inputs(60, lens, H, d)
    want = [[t.clone() for t in _everything(*x)] for x in (a, b)]
    for x, w in ((a, want[0]), (b, want[1])):
        for t, y in zip(_everything(*x), w):
            assert torch.equal(t, y)  # the same inputs give the same bits
    hold = [[t.clone() for t in a] for _ in range(2)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _everything(*hold[0])
    torch.cuda.synchronize()
    for h in hold:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_everything(*h))
        graphs.append(g)
    for order in ((0, 1), (1, 0)):
        for i, src in zip(order, (a, b)):
            for t, y in zip(hold[i], src):
                t.copy_(y)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i, w in zip(order, want):
            for t, y in zip(outs[i], w):
                assert torch.equal(t, y)


def test_on_other_streams_at_once():
    """Calls on two streams beside each other, none of them the current one."""
    sets = [_all_inputs(80 + 10 * i, [700, 33, 128], 2, 128) for i in range(2)]
    want = [[t.clone() for t in _everything(*x)] for x in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i, (x, s) in enumerate(zip(sets, streams)):
            Q, K, Vv, dO, cu, g, S0, dS = x
            O, lse = V.causal_attention(Q, K, Vv, cu, return_lse=True, stream=s)
            r = V.causal_attention_backward(Q, K, Vv, O, dO, lse, cu, stream=s)
            D, S = V.decay_attention(Q, K, Vv, g, cu, S0=S0, stream=s)
            b = V.decay_attention_backward(Q, K, Vv, dO, g, cu, S0=S0, dS=dS, stream=s)
            got[i] = [O, lse, *r.values(), D, S, *b.values()]
    torch.cuda.synchronize()
    for w, y in zip(want, got):
        for t, u in zip(w, y):
            assert torch.equal(t, u)


def test_prefix_arrays_that_are_wrong():
    """Starts beyond the tensor, falling or negative are clamped: wrong rows at most."""
    Q, K, Vv, dO, cu, g, S0, dS = _all_inputs(120, [40, 60], 2, 64)
    good = _everything(Q, K, Vv, dO, starts([40, 60], DEV), g, S0, dS)
    beyond = _everything(Q, K, Vv, dO, torch.tensor([0, 40, 1 << 30], dtype=torch.int32, device=DEV), g, S0, dS)
    for t, y in zip(good, beyond):
        assert torch.equal(t, y)
    for bad in ([-50, 40, 100], [60, 20, 90], [0, 100, 0], [1 << 30, -(1 << 30), 7]):
        _everything(Q, K, Vv, dO, torch.tensor(bad, dtype=torch.int32, device=DEV), g, S0, dS)
    L = 4096
    x = rand(1, L, 2, 64, unit=True).to(DEV)
    over = torch.tensor([0, L, 0, L, 0, L], dtype=torch.int32, device=DEV)  # overlapping long sequences
    V.decay_attention(x, x, x, g, over, S0=rand32(2, 5, 2, 64, 64).to(DEV))
    V.causal_attention(x, x, x, over)
    torch.cuda.synchronize()


def test_refusals_on_the_device():
    Q, K, Vv, dO, cu, g, S0, dS = _all_inputs(140, [30, 20], 2, 64)
    O, lse = V.causal_attention(Q, K, Vv, cu, return_lse=True)
    for call, match in [
        (lambda: V.causal_attention(Q, K.cpu(), Vv, cu), "is on cpu"),
        (lambda: V.causal_attention(Q.float(), K, Vv, cu), "dtype"),
        (lambda: V.causal_attention(Q, K[:, :, :32], Vv, cu), "shape"),
        (lambda: V.causal_attention(Q, K[:30], Vv[:30], cu), "give cu_k"),
        (lambda: V.causal_attention(Q, K, Vv, cu.long()), "dtype"),
        (lambda: V.causal_attention(Q, K, Vv, cu, cu_k=cu[:2]), "different numbers"),
        (lambda: V.causal_attention(Q, K, Vv, cu, k_len=torch.zeros(3, dtype=torch.int32, device=DEV)), "shape"),
        (lambda: V.causal_attention(Q[:, :1], K, Vv, cu), "no multiple"),
        (lambda: V.causal_attention(Q, K, Vv, cu, O=Q.transpose(1, 2)), "shape"),
        (lambda: V.causal_attention_backward(Q, K, Vv, O, dO, lse.half(), cu), "dtype"),
        (lambda: V.causal_attention_backward(Q, K, Vv, None, dO, lse, cu), "required"),
        (lambda: V.causal_attention_backward(Q, K, Vv, O, dO, lse, cu, out={"dQ": O}), "must hold"),
        (lambda: V.decay_attention(Q, K, Vv, g[:1], cu), "shape"),
        (lambda: V.decay_attention(Q, K, Vv, g.double(), cu), "dtype"),
        (lambda: V.decay_attention(Q, K, Vv, g, cu, S0=S0[:1]), "shape"),
        (lambda: V.decay_attention(Q, K, Vv, g, cu, S=S0.transpose(2, 3)), "contiguous"),
        (lambda: V.decay_attention_step(Q, K, Vv, g, S0), "shape"),
        (lambda: V.decay_attention_step(Q, K, Vv, g, None), "required"),
        (lambda: V.decay_attention_backward(Q, K, Vv, None, g, cu), "required"),
    ]:
        with pytest.raises(ValueError, match=match):
            call()
    for call in (lambda: V.causal_attention(Q, K, Vv, cu, scale=0.0),
                 lambda: V.causal_attention(Q[:, :, :32].contiguous(), K[:, :, :32].contiguous(),
                                            Vv[:, :, :32].contiguous(), cu),
                 lambda: V.decay_attention(Q, K, Vv, g, cu, scale=float("nan")),
                 lambda: V.decay_attention_backward(Q, K, Vv, dO, g, cu, dS=S0,
                                                    out={"dQ": O, "dK": O, "dV": O, "dS0": S0})):
        with pytest.raises(V.VDAError):
            call()
