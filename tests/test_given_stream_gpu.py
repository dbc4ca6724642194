"""Calls on another stream than the current one, with outputs and workspaces that the wrappers allocate."""
import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from hybrid_refs import D, gdn_inputs

pytestmark = pytest.mark.gpu


def _cases():
    x = gdn_inputs(300, 1, 2, seed=1)
    cu = torch.tensor([0, 200, 300], dtype=torch.int32)
    pool = (0.05 * torch.randn((8, 2, D, D), generator=torch.Generator().manual_seed(2))).cuda()
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    rows = [t[:24].contiguous() if t.shape[0] == 300 else t for t in x]
    one = [t[:6].contiguous() if t.shape[0] == 300 else t for t in x]
    pages = torch.randn((2, 40, 16, 2, D), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    table = torch.arange(36, dtype=torch.int32, device="cuda").view(6, 6)
    lens = torch.tensor([96, 1, 50, 0, 33, 70], dtype=torch.int32, device="cuda")
    q = torch.randn((6, 8, D), generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    g = torch.randn((300, 2, D), generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    bias = torch.zeros((2, D), device="cuda")
    z = x[0].expand(300, 2, D).contiguous()
    kw = dict(state_pool=pool, slot_ids=slots[:2], load_initial=True)
    cu_d = cu.cuda()
    return {
        "gdn_chunk_prefill": lambda s: kda.gdn_chunk_prefill(*x, cu_d, cu, **kw, stream=s),
        "gdn_recurrent_verify": lambda s: kda.gdn_recurrent_verify(*rows, pool, slots, 4, stream=s),
        "gdn_decode": lambda s: (kda.gdn_decode(*one, pool.clone() if s is None else _pool_on(pool, s), slots, stream=s),),
        "paged_attention": lambda s: kda.paged_attention(q, pages[0], pages[1], table, lens, stream=s)[:1],
        "chunk_prefill": lambda s: kda.chunk_prefill(z, z, x[2], g, x[4], x[5], bias, cu_d, cu, **kw, stream=s),
        "recurrent_verify": lambda s: kda.recurrent_verify(
            *(t[:24].contiguous() for t in (z, z, x[2], g, x[4])), x[5], bias, pool, slots, 4, stream=s),
    }


def _pool_on(pool, s):
    with torch.cuda.stream(s):
        return pool.clone()


@pytest.mark.parametrize("name", ["gdn_chunk_prefill", "gdn_recurrent_verify", "gdn_decode", "paged_attention", "chunk_prefill",
                                  "recurrent_verify"])
def test_outputs_are_the_given_streams(name):
    # The current stream still writes to memory that has just been given back to it; a call on another stream, whose results
    # are then read there, has to take other memory.
    call = _cases()[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    freed = [torch.empty_like(t) for t in want for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    for t in freed:
        t.fill_(7.0)
    del freed, t
    got = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
