"""Reads of tensor memory and the named barriers take whole warps, whichever product runs them. The code that the
streaming products share has them behind branches of single threads, so the warp is brought together again in front of
each, in every instantiation. Read from the kernels' source."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_mxfp4_bf16_gb300", "csrc")


def _source(path: str) -> str:
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _body(text: str, start: int) -> str:
    """The braces' contents from the first opening brace after `start` on."""
    at = text.index("{", start)
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at + 1:i]
    raise AssertionError("unbalanced braces")


def test_no_instantiation_goes_without_the_meeting_of_a_warp():
    paths = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))
    assert paths
    for path in paths:
        guarded = re.findall(r"if constexpr \([^;{}]*\)\s*__syncwarp", _source(path))
        assert not guarded, (os.path.basename(path), guarded)


def test_a_split_unit_brings_the_warp_together_before_what_takes_all_of_it():
    text = _source(os.path.join(CSRC, "stream_device.cuh"))
    body = _body(text, text.index("bool store_unit("))
    taking_all = [m for m in re.finditer(r"(?:load_tokens<kTermsPer>|named_barrier(?:_any)?)\(", body)]
    assert len(taking_all) == 6, "the pattern no longer finds what store_unit does"
    for m in taking_all:
        before = body[:m.start()]
        # a condition that is the same for the whole warp may stand between
        before = re.sub(r"(?:if constexpr \(!kLate\)|if \()\s*$", "", before).rstrip()
        assert before.endswith("__syncwarp();"), body[max(0, m.start() - 120):m.end()]
