"""Decayed linear attention whose sequences are cut into segments, as many as the workspace has
room for, beside ones that are not, against the float64 oracle."""
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
    assert V.sequence_poll() == V.VDA_OK


@pytest.mark.parametrize("H,d,lens", [
    (2, 64, [513] * 5),                              # a segment here is 512 tokens: two to each sequence
    (2, 128, [513, 1, 513, 0, 600, 512, 1025, 7]),
    (1, 64, [0, 513, 3, 512, 1024] * 8),             # more sequences than a warp counts by itself
    (1, 128, [2, 1, 0, 5] * 40 + [1025, 513]),       # and more than are sorted
])
def test_cut_and_uncut_sequences(H, d, lens):
    N, T = len(lens), sum(lens)
    Q, K, Vv, dO = rand(141, T, H, d, unit=True), rand(142, T, H, d, unit=True), rand(143, T, H, d), rand(144, T, H, d)
    S0, dS, g = rand32(145, N, H, d, d), rand32(146, N, H, d, d), slopes(H) / 64
    ref = po.decay_attention(f64(Q), f64(K), f64(Vv), f64(g), ranges(lens), f64(S0), 1.0, f64(dO), f64(dS))
    a, cu = [t.to(DEV) for t in (Q, K, Vv)], starts(lens, DEV)
    O, S = V.decay_attention(*a, g.to(DEV), cu, S0=S0.to(DEV))
    r = V.decay_attention_backward(*a, dO.to(DEV), g.to(DEV), cu, S0=S0.to(DEV), dS=dS.to(DEV))
    for n, x in (("O", O), ("dQ", r["dQ"]), ("dK", r["dK"]), ("dV", r["dV"])):
        bounded(f64(x), ref[n], ref["abs_" + n], n)
    # fp32 states: a step rounds once (2^-24), the sums over 128 tokens in steps of 16 for
    # three parts truncate 24 times (2^-23 each)
    for x, n in ((S, "S"), (r["dS0"], "dS0")):
        assert (np.abs(f64(x) - ref[n]) <= 2.0 ** -18 * ref["abs_" + n] + 1e-30).all()
