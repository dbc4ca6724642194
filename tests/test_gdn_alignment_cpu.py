"""Slot ids and sequence bounds of the gated delta rule that lie across words are refused on the host (fake device addresses;
never dereferenced)."""
import ctypes

import numpy as np
import pytest

from test_hybrid_cpu import FAKE, P, _decode, _head, _prefill, _verify, lib  # noqa: F401


@pytest.mark.parametrize("by", [1, 2, 3])
def test_words_apart(lib, by):  # noqa: F811
    assert _verify(lib, slots=FAKE + by) == 1
    assert _decode(lib, slots=FAKE + by) == 1
    for flags in (1, 2, 3):
        assert _prefill(lib, flags=flags, pool=FAKE, slots=FAKE + by, nslots=2) == 1
    head, hk, hv = _head()
    cu = np.array([0, 70], np.int32)
    size = lib.kda_gdn_prefill_workspace_size(70, 1, hv)
    assert lib.kda_gdn_chunk_prefill(*head, P(FAKE + by), cu.ctypes.data_as(ctypes.c_void_p), 1, hk, hv, None, 0, None, 0, P(FAKE),
                                     hv * 128, P(FAKE), P(FAKE), size, None) == 1
