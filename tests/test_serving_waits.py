"""CPU checks of how the chunk attention's warps wait. The waits are bounded by a time that every lane reads
for itself, and running out of it cannot be timed to fall between two lanes' readings, so the source is
checked: where a whole warp waits, its lanes vote."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "split_kv_decode_bsr_gb300", "csrc")


def _source(name):
    text = open(os.path.join(CSRC, name), encoding="utf-8").read()
    return re.sub(r"//[^\n]*", "", text)


def _barriers(text, call):
    """Names of the barriers that `call` is made on."""
    return set(re.findall(r"\b" + call + r"\(\s*&?(?:sh\.)?(\w+)", text))


def test_whole_warps_vote_where_they_wait():
    text = _source("chunk.cu")
    # waited for by whole warps: new items (K, V, MMA, softmax), free stages (K, V), products and the other slot's sums
    # (softmax)
    by_warps = {"item_full", "empty", "s_full", "o_full", "x_full"}
    assert by_warps <= _barriers(text, "mbar_wait_warp")
    assert not by_warps & _barriers(text, "mbar_wait")
    body = re.search(r"bool mbar_wait_warp\(.*?\{(.*?)\n\}", text, re.S).group(1)
    conditions = re.findall(r"if \((.*)\) (?:return true;|\{)", body)  # every way on or out is a vote
    assert len(conditions) == body.count("return") == 3
    assert all(re.match(r"__(all|any)_sync\(0xffffffffu, ", c) for c in conditions)


def test_a_wait_that_gives_up_is_heeded():
    """Nothing is written over a copy in flight, nor a stage passed on, after a wait that ran out. The outcome is
    dropped only where a role ends and its last copies or products are waited for, at most once more."""
    text = _source("chunk.cu")
    dropped = re.findall(r"(?:[;{}]|\bif \([^;{}]*\))\s*mbar_wait(?:_warp)?\(&sh\.(\w+)[^;]*;\s*([^;]*);", text)
    assert {name for name, _ in dropped} <= {"q_full", "full", "drain", "tail"}
    assert [after for name, after in dropped if name == "tail"] == ["break"]
