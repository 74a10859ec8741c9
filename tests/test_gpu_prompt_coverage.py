"""Every key, query and token of the prompt path counts once, at its place. All logits are 0
(or all pairs 1), and one tensor holds a single 1 in each channel, another row for each, moved
over the whole sequence: a row that a tile, share, block or ring slot leaves out, takes twice
or puts elsewhere changes a whole value."""
import pytest
import torch

from frame_level_delta_b200 import vda as V
from tests.prompt_cases import U, starts

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = dict(dtype=torch.bfloat16, device=DEV)


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    V.lib()


@pytest.fixture(autouse=True)
def _no_timeout():
    yield
    assert V.sequence_poll() == V.VDA_OK


def _ones(x, first, rows):
    """Row first + c of every sequence (its ``rows`` rows follow each other in x) has a 1 in channel c."""
    x = x.view(-1, rows, *x.shape[1:])
    for c in range(min(x.shape[-1], rows - first)):
        x[:, first + c, :, c] = 1


def _seen(nq, nk, first, d):
    """[nq, d]: query r sees key first + c; and the number of keys each sees."""
    r = torch.arange(nq, device=DEV)
    at = first + torch.arange(d, device=DEV)
    n = nk - nq + r + 1
    return (at < n[:, None]) & (at < nk), n.double()


FORMS = [  # name, query and key heads, d, queries, keys to a sequence, sequences: each form that sizes choose
    ("one_stream", 3, 1, 128, 300, 300, 5),
    ("one_stream_d64", 2, 2, 64, 700, 700, 2),
    ("two_streams", 2, 1, 128, 2600, 2600, 1),
    ("few_rows", 4, 1, 128, 1, 2500, 40),
    ("few_rows_d64", 2, 2, 64, 3, 1300, 3),
    ("few_rows_long", 1, 1, 64, 1, 9000, 1),
    ("few_tiles", 2, 2, 128, 100, 3000, 2),
]


@pytest.mark.parametrize("name,Hq,Hkv,d,nq,nk,N", FORMS, ids=[f[0] for f in FORMS])
def test_each_key_of_causal_attention(name, Hq, Hkv, d, nq, nk, N):
    """Each weight is 1 / (keys seen), its rounding and the output's are within U of it; rooms
    hold five more rows, of 1000."""
    room = nk + 5
    Q = torch.zeros(N * nq, Hq, d, **BF)
    K = torch.randn(N * room, Hkv, d, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(torch.bfloat16)
    cq, ck = starts([nq] * N, DEV), starts([room] * N, DEV)
    kl = torch.full((N,), nk, dtype=torch.int32, device=DEV)
    for first in range(0, nk, d):
        Vv = torch.zeros(N * room, Hkv, d, **BF)
        _ones(Vv, first, room)
        Vv.view(N, room, Hkv, d)[:, nk:] = 1000
        O = V.causal_attention(Q, K, Vv, cq, cu_k=ck, k_len=kl).double().view(N, nq, Hq, d)
        seen, n = _seen(nq, nk, first, d)
        off = (O * n[:, None, None] - seen.double()[:, None]).abs()
        assert (off <= seen.double()[:, None] * (U + 2.0 ** -14)).all(), first


GRADS = [
    ("one_stream", 3, 1, 128, 300, 300, 2),
    ("d64", 2, 2, 64, 333, 333, 2),
    ("more_keys", 4, 2, 128, 100, 700, 1),
    ("long", 1, 1, 128, 1500, 1500, 1),
]


@pytest.mark.parametrize("name,Hq,Hkv,d,nq,nk,N", GRADS, ids=[f[0] for f in GRADS])
def test_each_pair_of_the_gradients(name, Hq, Hkv, d, nq, nk, N):
    """With p = 1 / n, values +-1 in one channel and dO 1 in it, ds = p (v_j - o_r). Each term
    is rounded once and each result once (p itself is within 2^-13: its log-sum is fp32)."""
    G, s, tol = Hq // Hkv, 0.125, 2 * U + U * U + 2.0 ** -13
    cq, ck = starts([nq] * N, DEV), starts([nk] * N, DEV)
    zq, zk = torch.zeros(N * nq, Hq, d, **BF), torch.zeros(N * nk, Hkv, d, **BF)
    sign = zk.clone()
    sign.view(N, nk, Hkv, d)[:, 0::2, :, 0] = 1
    sign.view(N, nk, Hkv, d)[:, 1::2, :, 0] = -1
    up = zq.clone()
    up[..., 0] = 1
    v = sign.view(N, nk, Hkv, d)[0, :, 0, 0].double()

    def grads(Q, K, Vv, dO):
        O, lse = V.causal_attention(Q, K, Vv, cq, cu_k=ck, scale=s, return_lse=True)
        return O, V.causal_attention_backward(Q, K, Vv, O, dO, lse, cq, cu_k=ck, scale=s)

    for first in range(0, nk, d):  # dQ by keys
        K = zk.clone()
        _ones(K, first, nk)
        O, g = grads(zq, K, sign, up)
        seen, n = _seen(nq, nk, first, d)
        ve = torch.zeros(d, dtype=torch.float64, device=DEV)
        m = min(d, nk - first)
        ve[:m] = v[first:first + m]
        o = O.double().view(N, nq, Hq, d)[..., :1]
        want = s * seen.double()[:, None] / n[:, None, None] * (ve - o)
        got = g["dQ"].double().view(N, nq, Hq, d)
        assert ((got - want).abs() <= tol * want.abs()).all(), ("dQ", first)
    shift = nk - nq
    key = torch.arange(nk, device=DEV)
    for first in range(0, nq, d):  # dK and dV by queries
        at = first + torch.arange(d, device=DEV)
        live = at < nq
        pair = (key[:, None] <= shift + at) & live  # [nk, d]
        n = (shift + at + 1).double()
        one = zq.clone()
        _ones(one, first, nq)
        O, g = grads(one, zk, sign, up)
        o = O.double().view(N, nq, Hq, d)[:, at.clamp(max=nq - 1), :, 0].view(N, d, Hkv, G).sum(-1)  # [N, d, Hkv]
        want = s * pair.double()[:, None] / n * (G * v[:, None, None] - o.transpose(1, 2)[:, None])
        got = g["dK"].double().view(N, nk, Hkv, d)
        # (a group's terms are rounded each, and their sum may be smaller than they are)
        size = s * pair.double()[:, None] / n * 2 * G
        assert ((got - want).abs() <= tol * (want.abs() if G == 1 else size)).all(), ("dK", first)
        _, g = grads(zq, zk, sign, one)
        want = G * pair.double()[:, None] / n
        got = g["dV"].double().view(N, nk, Hkv, d)
        assert ((got - want).abs() <= tol * want).all(), ("dV", first)


@pytest.mark.parametrize("H,d,n,N", [(2, 128, 300, 3), (1, 64, 700, 2), (1, 128, 2500, 1), (2, 64, 1300, 2)])
def test_each_token_of_decay_attention(H, d, n, N):
    """A head that keeps everything, and pairs whose product is 1: every sum is of ones at
    different places, so every result is exact."""
    z, g, cu = torch.zeros(N * n, H, d, **BF), torch.zeros(H, device=DEV), starts([n] * N, DEV)
    e = z.clone()
    e[..., 0] = 1
    t = torch.arange(n, device=DEV)

    def check(x, m, what):
        assert (x.view(N, n, H, d) == m.to(x.dtype)[:, None]).all(), what

    for first in range(0, n, d):
        at = first + torch.arange(d, device=DEV)
        live = at < n
        past, behind = (at <= t[:, None]) & live, (at >= t[:, None]) & live
        one = z.clone()
        _ones(one, first, n)
        O, S = V.decay_attention(e, e, one, g, cu)
        check(O, past, "O")
        want = torch.zeros(N, H, d, d, device=DEV)
        want[..., 0] = live.float()
        assert torch.equal(S, want), "S"
        # dq_t = sum of (v.do) k over the past, dk_t and dv_t over what is behind it
        check(V.decay_attention_backward(e, one, e, e, g, cu)["dQ"], past, "dQ")
        r = V.decay_attention_backward(one, e, e, e, g, cu)
        check(r["dK"], behind, "dK")
        want = torch.zeros(N, H, d, d, device=DEV)
        want[..., 0, :] = live.float()
        assert torch.equal(r["dS0"], want), "dS0"
        check(V.decay_attention_backward(e, e, e, one, g, cu)["dV"], behind, "dV")
