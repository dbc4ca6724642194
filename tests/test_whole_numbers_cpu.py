"""Counts given to the calls beside the KDA layers are whole numbers; they are checked before any tensor."""
import numpy as np
import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from kda_linear_attention_bounded_gb300 import build as kbuild

Z = torch.zeros(3, dtype=torch.int32)


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


CALLS = {
    "verify": ("T", lambda n: kda.gdn_recurrent_verify(Z, Z, Z, Z, Z, Z, Z, Z, Z, n, out=Z, intermediate_states=Z, workspace=Z)),
    "paged": ("T", lambda n: kda.paged_attention(Z, Z, Z, Z, Z, n, out=Z, workspace=Z)),
    "tables": ("page_size", lambda n: kda.step_tables(Z, Z, Z, Z, n, cu_seqlens=Z, kv_lens=Z, positions=Z, slot_map=Z,
                                                      pages_used=Z, workspace=Z)),
}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("n", [2.9, 2.0, "16", None, np.float32(1), torch.tensor(1.5), [1]])
def test_what_is_no_whole_number_is_refused(call, n):
    name, f = CALLS[call]
    with pytest.raises(TypeError, match=f"{name}: expected a whole number"):
        f(n)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("n", [2 ** 31, -2 ** 31 - 1, 2 ** 70])
def test_what_is_out_of_range_is_refused(call, n):
    name, f = CALLS[call]
    with pytest.raises(ValueError, match=f"{name}: out of range"):
        f(n)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("n", [2, np.int64(2), torch.tensor(2), True])
def test_whole_numbers_are_taken(call, n):
    with pytest.raises(ValueError, match="expected a CUDA tensor"):   # (the next check)
        CALLS[call][1](n)


def test_sizes():
    with pytest.raises(TypeError):
        kda.paged_workspace_size(8, 2, 1.5)
    assert kda.paged_workspace_size(8, np.int64(2), 1) == kda.paged_workspace_size(8, 2)
