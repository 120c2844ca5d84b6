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


# -------------------------------------------------------------------------- requests sharing blocks
def shared_cache(lens, hq, hkv, d, dtype, bs, seed, extra):
    """Requests that all read the blocks of the longest one, from its first on."""
    c = ref.Cache([max(lens)], hq, hkv, d, dtype, bs, seed, extra=extra)
    c.lens = lens
    c.k, c.v = [c.k[0][:n] for n in lens], [c.v[0][:n] for n in lens]
    c.table, c.cu = c.table.expand(len(lens), -1).contiguous(), cu_seqlens(lens)
    return c


@pytest.mark.parametrize("lens,hq,hkv,d,dtype,bs,split,alibi", [
    ([1200, 1200, 960], 8, 2, 64, BF, 16, 0, False),
    ([1200, 1200, 960], 8, 2, 64, BF, 16, 64, True),
    ([800] * 50 + [1, 0, 799], 16, 2, 128, FP, 32, 128, False),   # fifty times the cache's slots
    ([3000, 2999, 17, 3000], 40, 2, 128, BF, 64, 0, True),
    ([500, 500], 4, 4, 256, FP, 16, 64, False),
])
def test_decode_paged_over_shared_blocks(lens, hq, hkv, d, dtype, bs, split, alibi):
    """Without a bound on the keys the workspace is sized by the cache's slots: the requests together
    hold more keys than that, and all of them count."""
    c = shared_cache(lens, hq, hkv, d, dtype, bs, 141, extra=1)
    assert sum(lens) > c.num_blocks * bs
    q = randn((len(lens), hq, d), 142, dtype)
    slopes = alibi_slope_values(hq) if alibi else None
    kc, vc, table, cu = c.gpu()
    gs = None if slopes is None else slopes.cuda()
    o, m, z, _ = ref.decode(c, q, d ** -0.5, slopes)
    size = mea.decode_workspace_size(len(lens), c.num_blocks * bs, hq, hkv, d, split)
    ws = torch.zeros(size + 4096, dtype=torch.uint8, device="cuda")
    ws[size:] = 77
    for kw in ({}, {"workspace": ws[:size]}, {"total_k_bound": sum(lens)}):
        out, lse = mea.decode_paged(q.cuda(), kc, vc, table, cu, max(lens), alibi_slopes=gs,
                                    scale=d ** -0.5, split_keys=split, **kw)
        ref.check_out(out.cpu(), lse.cpu(), o, m, z, dtype)
    assert bool((ws[size:] == 77).all())
    assert mea.device_error() == 0


# ---------------------------------------------------------------------------- outputs over inputs
def test_eviction_refuses_updates_in_place():
    """The new lengths over the old ones, the kept weights over the weights: refused, and nothing
    written."""
    c = ref.Cache([64, 48], 2, 2, 64, BF, 16, 161)
    kc, vc, table, cu = c.gpu()
    w = randn((2, 2, 64), 162, torch.float32, "cuda")
    ot = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    ko = torch.zeros((4, 16, 2, 64), dtype=BF, device="cuda")
    before = (cu.clone(), w.clone())
    for kw in ({"out_cu_seqlens_k": cu}, {"out_weights": w.view(-1)[:64].view(2, 2, 16)}):
        with pytest.raises(mea.MeaError) as e:
            mea.evict_paged(kc, vc, table, cu, 64, w, 16, 2, ot, out_k_cache=ko,
                            out_v_cache=ko.clone(), **kw)
        assert e.value.rc == mea._lib.MEA_ERR_SHAPE
    torch.cuda.synchronize()
    assert torch.equal(cu, before[0]) and torch.equal(w, before[1]) and not bool(ko.any())


# ---------------------------------------------------------------------------------------- no keys
def test_requests_without_any_keys():
    """A batch before its first token: outputs of rows that attend to nothing, no weights, no keys."""
    n, hq, hkv, d, bs = 3, 4, 2, 64, 16
    dev = {"device": "cuda"}
    kc = torch.full((4, bs, hkv, d), math.nan, dtype=BF, **dev)
    table = torch.full((n, 2), 1 << 30, dtype=torch.int32, **dev)
    cu, q = torch.zeros(n + 1, dtype=torch.int32, **dev), randn((n, hq, d), 171, BF, "cuda")
    w = torch.empty((n, hkv, 0), **dev)
    for prev in (None, w):
        out, lse, _ = mea.decode_paged_weights(q, kc, kc, table, cu, 0, w, prev_weights=prev)
        assert not bool(out.any()) and bool((lse == -math.inf).all())
    ko = torch.zeros((n, bs, hkv, d), dtype=BF, **dev)
    vo = torch.zeros_like(ko)
    ids = torch.arange(n, dtype=torch.int32, **dev).view(n, 1)
    kept, ow, ocu = mea.evict_paged(kc, kc, table, cu, 0, w, 8, 2, ids, out_k_cache=ko,
                                    out_v_cache=vo)
    assert bool((kept == -1).all()) and not bool(ow.any()) and not bool(ocu.any())
    assert not bool(ko.any()) and not bool(vo.any())
    sel = mea.select_blocks(q, torch.zeros((4, hkv, 2, d), dtype=BF, **dev), table, cu, 0, bs, 3)
    assert bool((sel == -1).all())
    mea.block_key_bounds(kc, table, cu, 0)
    for out, lse in (mea.decode_paged_selected(q, kc, kc, table, cu, sel),
                     mea.decode_paged(q, kc, kc, table, cu, 0),
                     mea.decode_tree_paged(q, kc, kc, table, cu, cu, 1, 0,
                                           torch.ones((n, 1), dtype=torch.int32, **dev),
                                           out=torch.zeros_like(q),
                                           lse=torch.full((hq, n), -math.inf, **dev))):
        assert not bool(out.any()) and bool((lse == -math.inf).all())
    none = torch.empty((0, hkv, d), dtype=BF, **dev)
    got = mea.attention_packed_weights(torch.empty((0, hq, d), dtype=BF, **dev), none,
                                       torch.empty((hq, 0), **dev), cu, cu, 0, 0)
    assert got.shape == (n, hkv, 0)
    assert mea.device_error() == 0


# ------------------------------------------------------------------------------- prompt's weights
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 256])
def test_prompt_weights_under_steep_slopes(d, causal):
    """Slopes under which distance terms are thousands of times the scores. The kernel's terms stay
    within 16.3 log2(e) * 16 = 376 of a counting weight's exponent: three roundings of values below
    512, half a step each, make 3 * 2^-16 ln 2 = 3.2e-5 at most, below the fp32 bound of 2^-14."""
    lens, hq, hkv = [700, 333], 4, 2
    q, k, v = make_qkv(lens, lens, hq, hkv, d, BF, 151)
    slopes = torch.tensor([16.3, 0.7, 5.1, 2.9])
    cu = cu_seqlens(lens)
    _, lse = mea.attention_packed(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), cu.cuda(), 700,
                                  causal=causal, alibi_slopes=slopes.cuda(), scale=d ** -0.5)
    got = mea.attention_packed_weights(q.cuda(), k.cuda(), lse, cu.cuda(), cu.cuda(), 700, 700,
                                       causal=causal, alibi_slopes=slopes.cuda(),
                                       scale=d ** -0.5).cpu()
    want = ref.prompt_weights(q, k, lse.cpu(), lens, lens, d ** -0.5, causal, slopes, 0, 700)
    for s, n in enumerate(lens):
        e = (got[s, :, :n].double() - want[s, :, :n]).abs()
        bound = ref.F32 * want[s, :, :n] + 1e-30
        assert bool((e <= bound).all()), float((e / bound).max())


def test_prompt_weights_of_more_columns_than_an_int_counts():
    """2^25 queries of 128 heads on one KV head are 2^32 (query, head) columns: each adds
    exp(0 - 0) = 1 to every key's weight (86 GB of zeros)."""
    lq, hq, d, lk = 1 << 25, 128, 8, 130
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB")
    q = torch.zeros((lq, hq, d), dtype=BF, device="cuda")
    lse = torch.zeros((hq, lq), device="cuda")
    k = torch.zeros((lk, 1, d), dtype=BF, device="cuda")
    w = mea.attention_packed_weights(q, k, lse, cu_seqlens([lq]).cuda(), cu_seqlens([lk]).cuda(),
                                     lq, lk).cpu()
    # (whole numbers: only the fp32 additions of the partial sums, up to 2^32, round)
    assert float((w.double() / (lq * hq) - 1).abs().max()) <= 148 * 2.0 ** -24
    assert mea.device_error() == 0


def steps_of(lens_q, lens_k, hq, hkv, d, causal, last, sms=148):
    """The kernel's schedule by its definition: steps per item of one head block, head blocks, and
    the equal ranges that the CTAs take."""
    r = hq // hkv
    p = 1
    while p < 128 and r % (2 * p) == 0:
        p *= 2
    kt, qt = (128 if d > 128 else 256), 128 // p
    items = []  # (Q tiles, head blocks) in the order of the line
    for lq, lk in zip(lens_q, lens_k):
        qw = max(0, lq - last) if last else 0
        for _ in range(hkv):
            for j in range(0, lk, kt):
                first = max(qw, j - (lk - lq)) if causal else qw
                items.append((max(-(-(lq - first) // qt), 1), r // p))
    total = sum(n * h for n, h in items)
    # (the host's bound on the steps sizes the grid)
    bound = len(lens_q) * hkv * -(-max(lens_k) // kt) * (r // p) * (-(-max(lens_q) // qt) + 1)
    return items, total, -(-total // min(bound, sms))


def prompt_weights_gpu(q, k, lse, lens_q, lens_k, scale, causal, slopes, last, width):
    """cache_reference.prompt_weights in 64 bits on the GPU, some rows at a time."""
    hq, hkv = q.shape[1], k.shape[1]
    out = torch.zeros(len(lens_q), hkv, width, dtype=torch.float64, device="cuda")
    qo = ko = 0
    for s, (lq, lk) in enumerate(zip(lens_q, lens_k)):
        j = torch.arange(lk, device="cuda")
        for i0 in range(max(0, lq - last) if last else 0, lq, 1024):
            i = torch.arange(i0, min(lq, i0 + 1024), device="cuda")
            pos = i + lk - lq
            for h in range(hq):
                x = scale * (q[qo + i, h].double() @ k[ko:ko + lk, h // (hq // hkv)].double().t())
                if slopes is not None:
                    x -= float(slopes[h]) * (pos[:, None] - j).abs()
                x -= lse[h, qo + i, None].double()
                if causal:
                    x.masked_fill_(j[None, :] > pos[:, None], -math.inf)
                out[s, h // (hq // hkv), :lk] += torch.exp(x).sum(0)
        qo += lq
        ko += lk
    return out.cpu()


@pytest.mark.parametrize("lens_q,lens_k,hq,hkv,d,dtype,causal,alibi,last", [
    ([3000, 2100, 5], [3000, 2100, 5], 16, 8, 64, BF, True, True, 0),
    ([3000, 2100, 5], [3000, 2100, 5], 16, 8, 128, BF, True, False, 0),
    ([3000, 2100, 5], [3000, 2100, 5], 16, 8, 128, FP, False, True, 0),
    ([2500, 130], [1700, 4000], 24, 2, 128, BF, True, True, 0),     # 12 heads a group: 3 blocks of 4
    ([1500, 0, 900], [2200, 300, 900], 36, 4, 80, FP, False, False, 0),  # 9 heads: 9 blocks of 1
    ([2600, 700], [2600, 700], 16, 4, 256, BF, True, True, 0),      # four score buffers
    ([1800, 999], [1800, 999], 12, 2, 200, FP, False, False, 0),
    ([200, 137, 256, 64] * 60, [200, 137, 256, 64] * 60, 8, 4, 64, BF, True, False, 0),
    ([600, 300] * 20, [2000, 1100] * 20, 32, 8, 128, BF, True, True, 100),
])
def test_prompt_weights_of_many_steps_a_cta(lens_q, lens_k, hq, hkv, d, dtype, causal, alibi, last):
    """Ranges of many steps: the join of the warpgroups, rings and queues that come round several
    times, items begun by one CTA and ended by another, head blocks that follow each other."""
    items, total, per = steps_of(lens_q, lens_k, hq, hkv, d, causal, last)
    nbuf = 4 if d > 128 else 2
    assert per > 2 * nbuf
    if items[0][1] > 1:  # a CTA's range crosses from one head block of an item to the next
        at, crossed = 0, False
        for n, hb in items:
            crossed |= any((at + n * b) % per for b in range(1, hb))
            at += n * hb
        assert crossed
    q, k, v = make_qkv(lens_q, lens_k, hq, hkv, d, dtype, 181)
    slopes = alibi_slope_values(hq) if alibi else None
    gs = None if slopes is None else slopes.cuda()
    q, k, v, cq, ck = q.cuda(), k.cuda(), v.cuda(), cu_seqlens(lens_q).cuda(), \
        cu_seqlens(lens_k).cuda()
    _, lse = mea.attention_packed(q, k, v, cq, ck, max(lens_q), causal=causal, alibi_slopes=gs,
                                  scale=d ** -0.5)
    width = max(lens_k) + 3
    w = torch.full((len(lens_q), hkv, width), 7.0, device="cuda")
    run = lambda: mea.attention_packed_weights(  # noqa: E731
        q, k, lse, cq, ck, max(lens_q), max(lens_k), causal=causal, alibi_slopes=gs,
        scale=d ** -0.5, last_queries=last, weights=w).cpu()
    got, again = run(), run()
    assert torch.equal(got, again)
    want = prompt_weights_gpu(q, k, lse, lens_q, lens_k, d ** -0.5, causal, slopes, last, width)
    for s, lk in enumerate(lens_k):
        e = (got[s, :, :lk].double() - want[s, :, :lk]).abs()
        bound = ref.F32 * want[s, :, :lk] + 1e-30
        assert bool((e <= bound).all()), float((e / bound).max())
        assert bool((got[s, :, lk:] == 7).all())
    assert mea.device_error() == 0


# ------------------------------------------------------------------------------ many short requests
def test_many_short_requests_cost_what_they_do_in_batches():
    """1024 requests of up to 600 keys in one call take no longer than in sixteen calls of 64: what a
    CTA does besides its own request does not grow with the batch."""
    n, hkv, d, bs, keep, part = 1024, 8, 64, 32, 128, 64
    lens = torch.randint(16, 601, (n,), generator=torch.Generator().manual_seed(201))
    nblk = [-(-int(x) // bs) for x in lens]
    table = torch.zeros((n, max(nblk)), dtype=torch.int32)
    at = 0
    for b, m in enumerate(nblk):
        table[b, :m] = torch.arange(at, at + m)
        at += m
    table = table.cuda()
    kc = torch.zeros((at, bs, hkv, d), dtype=BF, device="cuda")
    w = torch.rand((n, hkv, 600), device="cuda")
    per = keep // bs
    ot = torch.arange(n * per, dtype=torch.int32, device="cuda").view(n, per)
    ko = torch.zeros((n * per, bs, hkv, d), dtype=BF, device="cuda")
    bounds = torch.rand((at, hkv, 2, d), device="cuda").to(BF)
    q = torch.rand((n, hkv, d), device="cuda").to(BF)

    def step(a, b, cu):
        mea.evict_paged(kc, kc, table[a:b], cu, 600, w[a:b], keep, 8, ot[a:b], out_k_cache=ko,
                        out_v_cache=ko)
        mea.select_blocks(q[a:b], bounds, table[a:b], cu, 600, bs, 4)

    whole = cu_seqlens(lens.tolist()).cuda()
    parts = [cu_seqlens(lens[a:a + part].tolist()).cuda() for a in range(0, n, part)]
    calls = {"one": [(0, n, whole)],
             "many": [(i * part, (i + 1) * part, cu) for i, cu in enumerate(parts)]}
    times = {}
    for name, args in list(calls.items()) * 2:  # (the second time counts)
        start, end = torch.cuda.Event(True), torch.cuda.Event(True)
        torch.cuda.synchronize()
        start.record()
        for _ in range(3):
            for a in args:
                step(*a)
        end.record()
        torch.cuda.synchronize()
        times[name] = start.elapsed_time(end)
    assert times["one"] <= 1.5 * times["many"], times


def test_as_many_blocks_as_can_be_chosen_from():
    """50000 blocks of one request: the rank keys take all the shared memory there is."""
    n_blocks, bs, d, hq = 50000, 16, 256, 2
    length = n_blocks * bs - 3
    table = torch.randperm(n_blocks, generator=torch.Generator().manual_seed(211)).view(1, -1)
    bounds = randn((n_blocks, 1, 2, d), 212, FP, "cuda").sort(2).values
    q = randn((1, hq, d), 213, FP, "cuda")
    tab, cu = table.int().cuda(), cu_seqlens([length]).cuda()
    got = mea.select_blocks(q, bounds, tab, cu, length, bs, 777).cpu()
    x = q.double()[0]
    up, down = x.clamp_min(0).sum(0), x.clamp_max(0).sum(0)
    b = bounds[table[0].cuda(), 0].double()
    score = (b[:, 1] @ up + b[:, 0] @ down).float()
    score[0] = score[-1] = math.inf
    order = torch.sort(score, descending=True, stable=True).indices[:777].sort().values
    assert got[0, 0].tolist() == order.tolist()
    with pytest.raises(mea.MeaError):
        mea.select_blocks(q, bounds, torch.cat((tab, tab), 1), cu, length + 16, bs, 777)


# ------------------------------------------------------------------------------------- any scale
@pytest.mark.parametrize("scale", [-0.125, 0.0, 3.0])
@pytest.mark.parametrize("alibi", [False, True])
def test_scales_of_either_sign(scale, alibi):
    """Scales that are not positive turn the order of the scores round, or leave the bias alone."""
    lens, nq, hq, hkv, d, bs = [700, 129, 40], [9, 40, 1], 8, 2, 64, 16
    c = ref.Cache(lens, hq, hkv, d, FP, bs, 221)
    kc, vc, table, cu = c.gpu()
    slopes = alibi_slope_values(hq) if alibi else None
    gs = None if slopes is None else slopes.cuda()
    q, tq = randn((3, hq, d), 222, FP), randn((sum(nq), hq, d), 223, FP)
    every = torch.arange(44, dtype=torch.int32, device="cuda").expand(3, hkv, -1)
    w = torch.zeros((3, hkv, 700), device="cuda")
    o, m, z, want = ref.decode(c, q, scale, slopes)
    for out, lse in (mea.decode_paged_selected(q.cuda(), kc, vc, table, cu, every,
                                               alibi_slopes=gs, scale=scale),
                     mea.decode_paged_weights(q.cuda(), kc, vc, table, cu, 700, w,
                                              alibi_slopes=gs, scale=scale)[:2]):
        ref.check_out(out.cpu(), lse.cpu(), o, m, z, FP)
    for b, n in enumerate(lens):
        x = torch.stack(want[b])
        assert bool(((w.cpu()[b, :, :n].double() - x).abs() <= 2 * ref.F32 * x + 1e-30).all())
    masks = [torch.ones(n, n, dtype=torch.bool).tril() for n in nq]
    o, m, z = ref.tree(c, tq, nq, masks, scale, slopes)
    out, lse = mea.decode_tree_paged(tq.cuda(), kc, vc, table, cu_seqlens(nq).cuda(), cu, 40, 700,
                                     mea.tree_mask([list(range(-1, n - 1)) for n in nq]).cuda(),
                                     alibi_slopes=gs, scale=scale)
    ref.check_out(out.cpu(), lse.cpu(), o, m, z, FP)
    k, v = torch.cat(c.k), torch.cat(c.v)
    pq = randn((sum(lens), hq, d), 224, FP)
    cp = cu_seqlens(lens).cuda()
    _, lse = mea.attention_packed(pq.cuda(), k.cuda(), v.cuda(), cp, cp, 700, causal=True,
                                  alibi_slopes=gs, scale=scale)
    got = mea.attention_packed_weights(pq.cuda(), k.cuda(), lse, cp, cp, 700, 700, causal=True,
                                       alibi_slopes=gs, scale=scale).cpu()
    want = ref.prompt_weights(pq, k, lse.cpu(), lens, lens, scale, True, slopes, 0, 700)
    for s, n in enumerate(lens):
        assert bool(((got[s, :, :n].double() - want[s, :, :n]).abs() <=
                     ref.F32 * want[s, :, :n] + 1e-30).all())
    assert mea.device_error() == 0


# --------------------------------------------------------------------------------- a serving loop
def test_tokens_after_an_eviction():
    """Evict, append a token, decode with weights, and again: the kept weights go to the front of the
    next step's rows, the new key adds its own, and the next eviction goes by both."""
    total, hq, hkv, d, bs, keep, recent = [230, 60, 35], 8, 2, 64, 16, 40, 6
    n, rounds = len(total), 3
    c = ref.Cache([x + rounds for x in total], hq, hkv, d, BF, bs, 231)  # the later tokens' keys too
    kc, vc, table, _ = c.gpu()
    cu, max_k = cu_seqlens(total).cuda(), max(total)
    w = torch.rand((n, hkv, max_k), generator=torch.Generator().manual_seed(232)).cuda()
    old = w.cpu().double()
    keys = [[list(range(x)) for _ in range(hkv)] for x in total]
    per = -(-(keep + 1) // bs)
    for step in range(rounds):
        # (two sets of blocks, in turn: none is read and written by one eviction)
        ko = torch.full((n * per, bs, hkv, d), math.nan, dtype=BF, device="cuda")
        vo = torch.full_like(ko, math.nan)
        ot = torch.randperm(n * per, generator=torch.Generator().manual_seed(step)).view(n, per)
        ot = ot.int().cuda()
        kept, ow, ocu = mea.evict_paged(kc, vc, table, cu, max_k, w, keep, recent, ot,
                                        out_k_cache=ko, out_v_cache=vo)
        lens = [min(x if step == 0 else len(keys[b][0]), keep) for b, x in enumerate(total)]
        assert ocu.cpu().tolist() == cu_seqlens(lens).tolist()
        was, now = old, torch.zeros((n, hkv, keep + 1)).double()
        for b in range(n):
            for g in range(hkv):
                at = kept[b, g, :lens[b]].tolist()
                m = max(0, len(keys[b][g]) - recent)
                if len(keys[b][g]) > keep:
                    order = sorted(range(m), key=lambda t: (-float(w[b, g, t]), t))
                    assert at == sorted(order[:keep - recent]) + list(range(m, len(keys[b][g])))
                now[b, g, :lens[b]] = was[b, g, at]
                keys[b][g] = [keys[b][g][t] for t in at] + [total[b] + step]
            ko[ot[b, lens[b] // bs], lens[b] % bs] = c.k[b][total[b] + step].cuda()
            vo[ot[b, lens[b] // bs], lens[b] % bs] = c.v[b][total[b] + step].cuda()
        cu = cu_seqlens([x + 1 for x in lens]).cuda()
        kc, vc, table, max_k = ko, vo, ot, keep + 1
        w = torch.zeros((n, hkv, max_k), device="cuda")
        w[:, :, :keep] = ow
        q = randn((n, hq, d), 240 + step, BF)
        out, lse, _ = mea.decode_paged_weights(q.cuda(), kc, vc, table, cu, max_k, w,
                                               prev_weights=w, scale=0.125)
        o, m, z, p = ref.decode(c, q, 0.125, None, keys)
        ref.check_out(out.cpu(), lse.cpu(), o, m, z, BF)
        for b in range(n):
            now[b, :, :lens[b] + 1] += torch.stack(p[b])
        old = now
        # fp32: the weights' own bound in every round so far, and the additions' rounding
        assert bool(((w.cpu().double() - now).abs() <= (step + 2) * ref.F32 * now + 1e-30).all())
    assert mea.device_error() == 0
