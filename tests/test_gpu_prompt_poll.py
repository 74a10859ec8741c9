"""The prompt path's status word: a wait that gave up is reported once, by one poll."""
import threading

import pytest
import torch

from frame_level_delta_b200 import vda as V

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    V.lib()


def test_a_wait_that_gave_up_is_reported_once():
    assert V.sequence_poll() == V.VDA_OK
    assert V.selftest_sequence_wait(1000) == V.VDA_OK
    assert V.sequence_poll() == 6  # VDA_ERR_TIMEOUT
    assert V.sequence_poll() == V.VDA_OK


def test_one_of_several_polls_at_once_reports_it():
    """Each thread on a stream of its own; the word is the device's."""
    n, rounds = 4, 200
    streams = [torch.cuda.Stream() for _ in range(n)]
    got = [[None] * rounds for _ in range(n)]
    meet = threading.Barrier(n)

    def poll(i):
        for r in range(rounds):
            if i == 0:
                V.selftest_sequence_wait(100, stream=streams[0])
                streams[0].synchronize()
            meet.wait()
            got[i][r] = V.sequence_poll(stream=streams[i])
            meet.wait()

    threads = [threading.Thread(target=poll, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert [sorted(g[r] for g in got) for r in range(rounds)] == [[0] * (n - 1) + [6]] * rounds


def test_a_report_right_behind_a_poll_is_kept():
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(200):
        V.selftest_sequence_wait(10, stream=b)
        b.synchronize()
        assert V.sequence_poll(stream=a) == 6
        V.selftest_sequence_wait(10, stream=b)
        b.synchronize()
        assert V.sequence_poll(stream=a) == 6
    assert V.sequence_poll() == V.VDA_OK
