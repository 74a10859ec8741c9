"""The prompt path's calls from several threads at once, each on a stream of its own: they share
the remembered checks and the status word, and nothing else."""
import threading

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


def _inputs(seed, lens, H, d):
    T, N = sum(lens), len(lens)
    return [*(rand(seed + i, T, H, d, unit=i < 2).to(DEV) for i in range(4)), starts(lens, DEV), slopes(H).to(DEV),
            rand32(seed + 5, N, H, d, d).to(DEV), starts([1] * N, DEV)]


def _all(Q, K, Vv, dO, cu, g, S0, ones):
    N = S0.shape[0]
    O, lse = V.causal_attention(Q, K, Vv, cu, return_lse=True)
    r = V.causal_attention_backward(Q, K, Vv, O, dO, lse, cu)
    D, S = V.decay_attention(Q, K, Vv, g, cu, S0=S0)
    b = V.decay_attention_backward(Q, K, Vv, dO, g, cu, S0=S0, dS=S0)
    X = S.clone()
    s = V.decay_attention_step(Q[:N], K[:N], Vv[:N], g, X)
    return [O, lse, *r.values(), D, S, *b.values(), X, s, V.causal_attention(Q[:N], K, Vv, ones, cu_k=cu)]


def test_threads():
    sets = [_inputs(300 + 10 * i, lens, H, d) for i, (lens, H, d) in enumerate(
        [([300, 1, 128], 3, 128), ([1700, 40], 2, 64), ([300, 1, 128], 3, 128), ([20] * 40, 2, 64)])]
    want = [[t.clone() for t in _all(*x)] for x in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(15):
                got = _all(*sets[i])
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [] and V.sequence_poll() == V.VDA_OK
