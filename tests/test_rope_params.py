"""Copies of a Rope, as those of the model that holds it: their parameters point to their own speeds."""

import copy
import ctypes as C
import pickle

import pytest

import split_kv_decode_bsr_gb300 as sta


def _speeds(rope, n):
    at = sta._RopeParams.from_buffer_copy(rope.packed()).freqs
    return at, [C.c_double.from_address(at + 8 * i).value for i in range(n)]


@pytest.mark.parametrize("made", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))])
@pytest.mark.parametrize("read", [False, True])  # the struct has been asked for: it may have been changed since
def test_copies_hold_their_own_speeds(made, read):
    freqs = [0.5, 0.25, 2.0, -1.0]
    rope = sta.Rope(8, interleaved=True, mscale=1.25, freqs=freqs)
    if read:
        rope.struct.mscale = 1.5
    two = made(rope)
    at, values = _speeds(two, 4)
    assert at == C.addressof(two._freqs) and values == freqs
    assert two.struct.freqs == at
    assert two.rot_dim == 8 and two.struct.layout == sta.STA_ROPE_INTERLEAVED and two.struct.mscale == (1.5 if read else 1.25)
    assert _speeds(rope, 4)[0] == C.addressof(rope._freqs)


@pytest.mark.parametrize("made", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))])
def test_copies_without_speeds_of_their_own(made):
    rope = sta.Rope(64, base=500000.0, scaling="linear", factor=4.0)
    assert made(rope).packed() == rope.packed() and made(rope).struct.freqs is None
    rope.struct.factor = 8.0
    assert made(rope).packed() == rope.packed() and made(rope).struct.factor == 8.0
