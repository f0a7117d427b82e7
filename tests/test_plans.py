"""CPU checks of the attention's plans where there is next to nothing to plan."""

import numpy as np
import pytest

import split_kv_decode_bsr_gb300 as sta
from split_kv_decode_bsr_gb300 import build as sta_build

I32 = np.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    sta_build.build()


@pytest.mark.parametrize("kv,window", [((0, 0, 0, 0), None), ((0, 1, 3, 12), (5, 9)), ((0, 0, 0, 7), (-1, -1)), ((0, 1, 2, 300), None)])
@pytest.mark.parametrize("d", [64, 128])
def test_new_tokens_that_see_no_key(kv, window, d):
    # empty sequences, windows ahead of every token: no key tile for any request, or for some
    q = np.array([0, 1, 2, 5], I32)
    pattern = None if window is None else sta.MaskSource.pattern(causal=True, win_lo=window[0], win_hi=window[1])
    for splits in (0, 1, 7):
        need = sta.chunk_workspace_bytes(q, np.array(kv, I32), 3, 8, 2, d, pattern=pattern, num_splits=splits)
        assert need == 256 if splits < 7 else need > 256  # not cut, or cut as asked
    assert sta.chunk_workspace_bytes(np.zeros(4, I32), np.array(kv, I32), 3, 8, 2, d) == 256  # no new token


def test_prefixes_with_as_few_tokens_as_there_can_be():
    for new in ((1, 1, 1), (0, 1, 1), (0, 0, 1), (0, 0, 0)):
        q = np.concatenate([[0], np.cumsum(new)]).astype(I32)
        for prefix in (0, 1, 16):
            kv = np.concatenate([[0], np.cumsum(prefix + np.array(new))]).astype(I32)
            for splits in (0, 1, 1024):
                for Hq, Hkv in ((1, 1), (128, 1), (8, 8), (40, 20)):
                    assert sta.prefix_workspace_bytes(q, kv, 3, [0, 3], [prefix], Hq, Hkv, 64, 1, splits) >= 256
