"""The bound that the accuracy tests hold final states to lies between the kernels' roundings and coarser ones."""
import pytest
import torch

from gdn_rounding import final_states
from hybrid_refs import gdn_inputs, gdn_reference, rel_l2
from test_gdn_accuracy_gpu import STATES, state_bound

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("lens,a_mean", STATES)
def test_bound_tells_roundings_apart(lens, a_mean):
    x = gdn_inputs(sum(lens), 2, 4, seed=len(lens) + sum(lens), a_mean=a_mean, device="cpu")
    _, _, ref = gdn_reference(x, lens, keep=False)
    assert rel_l2(final_states(x, lens), ref) <= 1e-12
    bound = state_bound(x, lens)
    ours, coarse = final_states(x, lens, BF16, FP16), final_states(x, lens, BF16, BF16)
    for n in range(len(lens)):
        for h in range(4):
            assert rel_l2(ours[n, h], ref[n, h]) <= bound[n][h], (n, h)
            assert rel_l2(coarse[n, h], ref[n, h]) > bound[n][h], (n, h)
