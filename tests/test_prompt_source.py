"""Orders between threads that the prompt path's kernels have to state in their source,
because no run shows their absence for certain."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "frame_level_delta_b200", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _after_zeroing(text):
    """For each run of zero_row calls: what follows the fence behind it, without closing
    braces and fences of the tensor cores."""
    found = []
    for m in re.finditer(r"zero_row\([^;]*;(?:[\s}]|\w+::zero_row\([^;]*;)*?\s*fence_proxy_async_smem\(\);", text):
        rest = text[m.end():]
        found.append(re.sub(r"^(?:\s|\}|tc_fence_before\(\);)*", "", rest))
    return found


@pytest.mark.parametrize("name,places", [("causal_attn_tc.cu", 1), ("causal_attn_bwd_tc.cu", 3), ("decay_attn_tc.cu", 2)])
def test_zeroed_rows_are_ordered_before_their_warps_signal(name, places):
    """Every lane zeroes a row behind the sequence and fences its own stores; one lane then
    tells the issuing warp. All lanes have to meet in between on every way there, so the
    meeting is the next thing behind the fence, outside any branch (set_up meets the CTA)."""
    follow = _after_zeroing(_code(name))
    assert len(follow) == places
    for f in follow:
        assert f.startswith(("__syncwarp();", "seq::set_up(")), f[:80]
