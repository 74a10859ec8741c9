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
