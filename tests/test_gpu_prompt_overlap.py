"""Calls of the prompt path whose outputs share memory with something else are refused; outputs
that only lie between an input's rows are not."""
import pytest
import torch

from frame_level_delta_b200 import vda as V
from tests.prompt_cases import rand, rand32, slopes, starts

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    V.lib()


def test_shared_memory_is_refused_and_neighbours_are_not():
    H, d, lens = 2, 64, [70, 30]
    T, N = sum(lens), len(lens)
    cu, g = starts(lens, DEV), slopes(H).to(DEV)
    joint = rand(1, T, 4 * H, d, unit=True).to(DEV)
    Q, K, Vv, O = (joint[:, i * H:(i + 1) * H] for i in range(4))
    S0 = rand32(2, N, H, d, d).to(DEV)
    keep = joint.clone()
    want, lse = V.causal_attention(Q, K, Vv, cu, return_lse=True)
    V.causal_attention(Q, K, Vv, cu, O=O)
    assert torch.equal(O, want) and torch.equal(joint[:, :3 * H], keep[:, :3 * H])
    want_l, want_S = V.decay_attention(Q, K, Vv, g, cu, S0=S0)
    S = S0.clone()
    V.decay_attention(Q, K, Vv, g, cu, S0=S, S=S, O=O)
    assert torch.equal(O, want_l) and torch.equal(S, want_S) and torch.equal(joint[:, :3 * H], keep[:, :3 * H])
    one = V.decay_attention_step(Q[:N], K[:N], Vv[:N], g, S0.clone())
    V.decay_attention_step(Q[:N], K[:N], Vv[:N], g, S0.clone(), O=O[:N])
    assert torch.equal(O[:N], one)
    dO = rand(3, T, H, d).to(DEV)
    q, k, v = (t.contiguous() for t in (Q, K, Vv))
    new = lambda: {n: torch.empty_like(q) for n in ("dQ", "dK", "dV")}
    half = torch.empty(2 * T, H, d, dtype=torch.bfloat16, device=DEV)
    before = joint.clone()
    for call in (lambda: V.causal_attention(Q, K, Vv, cu, O=Q),
                 lambda: V.causal_attention(Q, K, Vv, cu, O=joint[:, H // 2:H // 2 + H]),
                 lambda: V.causal_attention(half[:T], k, v, cu, O=half[T // 2:T // 2 + T]),
                 lambda: V.causal_attention_backward(q, k, v, want, dO, lse, cu, out={**new(), "dQ": q}),
                 lambda: V.causal_attention_backward(q, k, v, want, dO, lse, cu, out=dict.fromkeys(("dQ", "dK", "dV"), half[:T])),
                 lambda: V.decay_attention(Q, K, Vv, g, cu, O=Vv),
                 lambda: V.decay_attention_step(Q[:N], K[:N], Vv[:N], g, S0, O=K[:N]),
                 lambda: V.decay_attention_backward(q, k, v, dO, g, cu, out={**new(), "dV": dO})):
        with pytest.raises(V.VDAError):
            call()
    assert torch.equal(joint, before)
