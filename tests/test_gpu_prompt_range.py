"""Decayed linear attention where states, tokens and decays lie far apart in size, against the
float64 oracle. The bounds are relative to what a result is made of, so they hold at any size."""
import numpy as np
import pytest
import torch

from frame_level_delta_b200 import vda as V
from oracle import prompt_oracle as po
from tests.prompt_cases import bounded, f64, rand, rand32, ranges, starts

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


def _compare(lens, ld, d, token, state):
    """Forward and gradients with Q, K, V and dO of the size ``token``, S0 and dS of ``state``."""
    H, T, N = len(ld), sum(lens), len(lens)
    Q, K, Vv, dO = (rand(121 + i, T, H, d, scale=token) for i in range(4))
    S0, dS = rand32(125, N, H, d, d) * state, rand32(126, N, H, d, d) * state
    ld = torch.tensor(ld)
    ref = po.decay_attention(f64(Q), f64(K), f64(Vv), f64(ld), ranges(lens), f64(S0), 1.0, f64(dO), f64(dS))
    a, cu = [t.to(DEV) for t in (Q, K, Vv)], starts(lens, DEV)
    O, _ = V.decay_attention(*a, ld.to(DEV), cu, S0=S0.to(DEV))
    r = V.decay_attention_backward(*a, dO.to(DEV), ld.to(DEV), cu, S0=S0.to(DEV), dS=dS.to(DEV))
    for n, x in (("O", O), ("dQ", r["dQ"]), ("dK", r["dK"]), ("dV", r["dV"])):
        bounded(f64(x), ref[n], ref["abs_" + n], n)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("state", [2.0 ** 70, 2.0 ** 110])
def test_a_state_far_above_the_tokens_is_forgotten_at_its_rate(state, d):
    """From a head that takes 128 tokens to forget such a state to one that keeps nothing."""
    _compare([200, 1, 128], [-0.3, -0.6, -1.5, -9.0, -44.0, -60.0, -90.0, -250.0, float("-inf")], d, 1.0, state)


@pytest.mark.parametrize("d", [64, 128])
def test_nothing_is_kept_at_minus_infinity(d):
    """A token's own term alone, bit for bit, whatever the state."""
    lens, H = [150, 40], 2
    Q, K, Vv = (rand(131 + i, sum(lens), H, d).to(DEV) for i in range(3))
    ld, cu = torch.full((H,), float("-inf"), device=DEV), starts(lens, DEV)
    S0 = (rand32(134, len(lens), H, d, d) * 2.0 ** 120).to(DEV)
    O, S = V.decay_attention(Q, K, Vv, ld, cu, S0=S0)
    O0, S1 = V.decay_attention(Q, K, Vv, ld, cu)
    assert torch.equal(O, O0) and torch.equal(S, S1)


@pytest.mark.parametrize("d", [64, 128])
def test_outputs_far_above_one(d):
    """Products near 2^90 in heads from slow to fast."""
    _compare([200, 128], [-1e-3, -0.17, -0.2, -0.34, -0.36, -1.0, -20.0], d, 2.0 ** 27, 2.0 ** 40)
