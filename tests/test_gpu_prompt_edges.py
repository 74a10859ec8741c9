"""Calls at the edges of the prompt path's ranges, against the float64 oracle."""
import numpy as np
import pytest
import torch

from frame_level_delta_b200 import vda as V
from oracle import prompt_oracle as po
from tests.prompt_cases import bounded, f64, rand, rand32, ranges, starts

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    V.lib()


@pytest.fixture(autouse=True)
def _no_timeout():
    yield
    assert V.sequence_poll() == V.VDA_OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [-0.4, -1.0, -3.0])
def test_large_values_in_heads_that_forget_fast(g, d):
    """Outputs near 2^32 (keys that meet their own query at 2^6 a channel) where a chunk's
    decay falls far below what fp32 holds. The bounds are relative, so they hold at any size."""
    H, lens = 2, [200, 128]
    T = sum(lens)
    K, Vv, dO = rand(61, T, H, d, scale=64.0), rand(62, T, H, d, scale=1024.0), rand(63, T, H, d, scale=1024.0)
    Q = K.clone()
    S0, dS = rand32(64, len(lens), H, d, d), rand32(65, len(lens), H, d, d)
    ld = torch.full((H,), g)
    ref = po.decay_attention(f64(Q), f64(K), f64(Vv), f64(ld), ranges(lens), f64(S0), 1.0, f64(dO), f64(dS))
    a = [t.to(DEV) for t in (Q, K, Vv)]
    O, _ = V.decay_attention(*a, ld.to(DEV), starts(lens, DEV), S0=S0.to(DEV))
    bounded(f64(O), ref["O"], ref["abs_O"], "O")
    r = V.decay_attention_backward(*a, dO.to(DEV), ld.to(DEV), starts(lens, DEV), S0=S0.to(DEV), dS=dS.to(DEV))
    for n in ("dQ", "dK", "dV"):
        bounded(f64(r[n]), ref[n], ref["abs_" + n], n)
