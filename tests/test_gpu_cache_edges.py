"""The paged-cache operators where calls follow each other closely, at sizes that take the longer
paths, and with arguments at the edge of what their documentation allows."""
import math

import pytest
import torch

import cache_reference as ref
import memory_efficient_attention_b200 as mea
from mea_workloads import alibi_slope_values, cu_seqlens, make_qkv, randn

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


# ---------------------------------------------------------------------- calls close to each other
@pytest.mark.parametrize("n,length", [(1, 3000), (5, 700)])
def test_lists_and_queries_rewritten_between_calls(n, length):
    """Every call sees what the kernel just before it on the stream wrote, be it the block choice or
    the caller's own copy: as with a wait for the GPU between the two."""
    hq, hkv, d, bs, steps = 8, 2, 128, 16, 12
    c = ref.Cache([length - 37 * b for b in range(n)], hq, hkv, d, BF, bs, 101)
    kc, vc, table, cu = c.gpu()
    bounds = mea.block_key_bounds(kc, table, cu, c.max)
    qs = [randn((n, hq, d), 102 + i, BF, "cuda") for i in range(steps)]
    lists = [torch.randint(0, -(-c.max // bs), (n, hkv, 7), device="cuda", dtype=torch.int32,
                           generator=torch.Generator("cuda").manual_seed(i)) for i in range(steps)]
    weights = [randn((n, hkv, c.max), 130 + i, torch.float32, "cuda") for i in range(steps)]
    ot = torch.arange(n * 4, dtype=torch.int32, device="cuda").view(n, 4)

    def run(wait):
        q, w = torch.empty_like(qs[0]), torch.empty_like(weights[0])
        sel = torch.empty_like(lists[0])
        kept = torch.empty((n, hkv, 60), dtype=torch.int32, device="cuda")
        ko = torch.zeros((n * 4, bs, hkv, d), dtype=BF, device="cuda")
        vo = torch.zeros_like(ko)
        outs = []
        for i in range(steps):
            q.copy_(qs[i])
            wait()
            mea.select_blocks(q, bounds, table, cu, c.max, bs, 7, selected=sel)
            wait()
            outs += mea.decode_paged_selected(q, kc, vc, table, cu, sel, scale=0.1)
            sel.copy_(lists[i])
            wait()
            outs += mea.decode_paged_selected(q, kc, vc, table, cu, sel, scale=0.1)
            w.copy_(weights[i])
            wait()
            outs += mea.evict_paged(kc, vc, table, cu, c.max, w, 60, 5, ot, out_k_cache=ko,
                                    out_v_cache=vo, kept=kept)[1:]
            outs += [kept.clone(), ko.clone(), vo.clone()]
        torch.cuda.synchronize()
        return outs

    for a, b in zip(run(torch.cuda.synchronize), run(lambda: None)):
        assert torch.equal(a, b)
    assert mea.device_error() == 0
