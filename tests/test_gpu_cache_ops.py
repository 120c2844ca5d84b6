"""Operators on a paged K/V cache against their 64-bit forms (tests/cache_reference.py): key ranges,
block choice, decode over chosen blocks, decode and prompt attention weights, eviction, and the
tree attention; then a run of them together."""
import math

import pytest
import torch

import cache_reference as ref
import memory_efficient_attention_b200 as mea
from mea_workloads import alibi_slope_values, cu_seqlens, make_qkv, randn

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def slopes_of(hq, alibi):
    return alibi_slope_values(hq) if alibi else None


def gpu(t):
    return None if t is None else t.cuda()


# ------------------------------------------------------------------------------------ key ranges
@pytest.mark.parametrize("lens,hkv,d,dtype,bs", [
    ([1], 1, 8, FP, 16),
    ([0, 17, 64, 33], 2, 64, BF, 16),
    ([200, 1, 129], 8, 128, FP, 32),
    ([500, 0, 77], 3, 136, BF, 64),
    ([385, 191], 2, 256, BF, 192),
])
def test_key_bounds(lens, hkv, d, dtype, bs):
    c = ref.Cache(lens, hkv, hkv, d, dtype, bs, 11)
    want, used = ref.block_bounds(c)
    kc, _, table, cu = c.gpu()
    before = randn(tuple(want.shape), 5, dtype)
    got = mea.block_key_bounds(kc, table, cu, c.max, bounds=before.cuda().clone()).cpu()
    assert torch.equal(got[used], want[used])
    assert torch.equal(got[~used], before[~used])
    # Only the blocks that hold keys from first_key on.
    first = torch.tensor([max(0, n - 1 - bs) for n in lens], dtype=torch.int32)
    part = mea.block_key_bounds(kc, table, cu, c.max, first_key=first.cuda(),
                                bounds=before.cuda().clone()).cpu()
    touched = torch.zeros_like(used)
    for b, n in enumerate(lens):
        for j in range(int(first[b]) // bs, -(-n // bs)):
            touched[int(c.table[b, j])] = True
    assert torch.equal(part[touched], want[touched])
    assert torch.equal(part[~touched], before[~touched])


def test_key_bounds_keep_a_nan_key():
    c = ref.Cache([20], 1, 1, 16, BF, 16, 3)
    kc, _, table, cu = c.gpu()
    kc[int(c.table[0, 1]), 2, 0, 5] = math.nan
    got = mea.block_key_bounds(kc, table, cu, 20).cpu()
    bad = torch.isnan(got)
    assert bool(bad[int(c.table[0, 1]), 0, :, 5].all()) and int(bad.sum()) == 2


# ---------------------------------------------------------------------------------- block choice
@pytest.mark.parametrize("lens,hq,hkv,d,dtype,bs,n_select,n_first,n_last", [
    ([1], 1, 1, 8, FP, 16, 1, 1, 1),
    ([0, 17, 300, 1000], 8, 2, 64, BF, 16, 5, 1, 1),
    ([700, 40], 6, 2, 80, FP, 32, 3, 0, 0),
    ([2000, 129, 64], 12, 1, 128, BF, 16, 40, 2, 3),
    ([4000], 8, 8, 40, FP, 16, 17, 0, 1),
    ([900, 1500], 8, 4, 256, BF, 16, 9, 1, 2),
    ([600], 4, 2, 136, FP, 16, 2, 3, 3),      # the forced blocks alone are more than asked for
    ([20000], 4, 1, 128, BF, 16, 64, 1, 1),   # a cluster of CTAs
])
def test_select_blocks(lens, hq, hkv, d, dtype, bs, n_select, n_first, n_last):
    c = ref.Cache(lens, hq, hkv, d, dtype, bs, 21)
    q = randn((len(lens), hq, d), 22, dtype)
    bounds, _ = ref.block_bounds(c)
    _, _, table, cu = c.gpu()
    got = mea.select_blocks(q.cuda(), bounds.cuda(), table, cu, c.max, bs, n_select,
                            n_first=n_first, n_last=n_last).cpu()
    want = ref.choose(c, q, bounds, n_select, n_first, n_last)
    for b in range(len(lens)):
        for g in range(hkv):
            row = want[b][g] + [-1] * (n_select - len(want[b][g]))
            assert got[b, g].tolist() == row


def test_select_blocks_ties_and_nan():
    """Equal scores go to the lower index; a NaN range ranks above every score."""
    c = ref.Cache([16 * 40], 2, 1, 64, BF, 16, 1)
    q = torch.ones((1, 2, 64), dtype=BF)
    bounds = torch.ones((c.num_blocks, 1, 2, 64), dtype=BF)
    _, _, table, cu = c.gpu()
    got = mea.select_blocks(q.cuda(), bounds.cuda(), table, cu, c.max, 16, 7, n_first=0, n_last=0)
    assert got.cpu()[0, 0].tolist() == list(range(7))
    bounds[int(c.table[0, 30]), 0, 1, 3] = math.nan
    bounds[int(c.table[0, 25]), 0, 1, 3] = math.inf
    got = mea.select_blocks(q.cuda(), bounds.cuda(), table, cu, c.max, 16, 3, n_first=0, n_last=1)
    assert got.cpu()[0, 0].tolist() == [25, 30, 39]


@pytest.mark.parametrize("dtype,factor", [(BF, 1e30), (BF, 1e-30), (FP, 3e4), (FP, 1e-6)])
def test_select_blocks_extreme_queries(dtype, factor):
    """Queries whose sums leave the range of fp32 products, or of 16 bits, change nothing in the choice's
    definition."""
    c = ref.Cache([900, 3000], 8, 2, 64, dtype, 16, 23)
    q = (randn((2, 8, 64), 24, torch.float32) * factor).clamp(-6e4, 6e4).to(dtype) \
        if dtype == FP else (randn((2, 8, 64), 24, torch.float32) * factor).to(dtype)
    bounds, _ = ref.block_bounds(c)
    if factor > 1e20:
        bounds = (bounds.float() * 1e8).to(dtype)
    _, _, table, cu = c.gpu()
    got = mea.select_blocks(q.cuda(), bounds.cuda(), table, cu, c.max, 16, 21).cpu()
    want = ref.choose(c, q, bounds, 21, 1, 1)
    for b in range(2):
        for g in range(2):
            assert got[b, g].tolist() == want[b][g]


def test_select_blocks_many_near_the_cut():
    """More blocks within the first scores' error than a list holds: all are decided in 64 bits."""
    c = ref.Cache([16 * 300], 4, 1, 128, BF, 16, 25)
    q = randn((1, 4, 128), 26, BF)
    bounds = randn((1, 1, 2, 128), 27, BF).expand(c.num_blocks, -1, -1, -1).clone()
    # Blocks differ in one column, by one rounding step of a value that hardly counts.
    pos = torch.randperm(300, generator=torch.Generator().manual_seed(28))
    for j in range(300):
        bounds[int(c.table[0, j]), 0, 1, 5] = 2.0 ** -12 * (1 + int(pos[j]) % 100 / 128)
    _, _, table, cu = c.gpu()
    got = mea.select_blocks(q.cuda(), bounds.cuda(), table, cu, c.max, 16, 50, n_first=0,
                            n_last=2).cpu()
    assert got[0, 0].tolist() == ref.choose(c, q, bounds, 50, 0, 2)[0][0]


# --------------------------------------------------------------------- decode over chosen blocks
@pytest.mark.parametrize("lens,hq,hkv,d,dtype,bs,n_select,alibi", [
    ([1], 1, 1, 8, FP, 16, 1, False),
    ([0, 17, 300, 1000], 8, 2, 64, BF, 16, 5, True),
    ([700, 40], 6, 2, 80, FP, 32, 9, False),
    ([2000, 129, 64], 12, 1, 128, BF, 16, 40, True),
    ([900, 1500], 8, 4, 256, BF, 64, 9, False),
    ([1000, 192], 40, 2, 128, FP, 192, 4, True),
    ([5000] * 40, 8, 4, 64, FP, 16, 33, False),
])
def test_decode_selected(lens, hq, hkv, d, dtype, bs, n_select, alibi):
    c = ref.Cache(lens, hq, hkv, d, dtype, bs, 31)
    n = len(lens)
    q, slopes = randn((n, hq, d), 32, dtype), slopes_of(hq, alibi)
    # Any order, gaps in the list, entries that name no block.
    gen = torch.Generator().manual_seed(7)
    sel = torch.full((n, hkv, n_select), -1, dtype=torch.int32)
    keys = []
    for b, length in enumerate(lens):
        nblk = -(-length // bs)
        keys.append([])
        for g in range(hkv):
            pick = torch.randperm(nblk, generator=gen)[:max(1, n_select - 1)].tolist()
            if g % 2:
                pick = sorted(pick)
            at = torch.randperm(n_select, generator=gen)[:len(pick)].sort().values
            sel[b, g, at] = torch.tensor(pick, dtype=torch.int32)
            if g == 0 and len(pick) < n_select:
                free = [i for i in range(n_select) if i not in at.tolist()]
                sel[b, g, free[0]] = nblk + 3
            keys[-1].append([t for j in pick for t in range(j * bs, min(length, (j + 1) * bs))])
    kc, vc, table, cu = c.gpu()
    out, lse = mea.decode_paged_selected(q.cuda(), kc, vc, table, cu, sel.cuda(),
                                         alibi_slopes=gpu(slopes), scale=d ** -0.5)
    o, m, z, _ = ref.decode(c, q, d ** -0.5, slopes, keys)
    ref.check_out(out.cpu(), lse.cpu(), o, m, z, dtype)
    assert mea.device_error() == 0


def test_decode_selected_counts_a_block_twice():
    c = ref.Cache([100], 2, 1, 64, BF, 16, 41)
    q = randn((1, 2, 64), 42, BF)
    kc, vc, table, cu = c.gpu()
    sel = torch.tensor([[[3, 1, 3]]], dtype=torch.int32)
    keys = [[list(range(48, 64)) + list(range(16, 32)) + list(range(48, 64))]]
    out, lse = mea.decode_paged_selected(q.cuda(), kc, vc, table, cu, sel.cuda(), scale=0.125)
    o, m, z, _ = ref.decode(c, q, 0.125, None, keys)
    ref.check_out(out.cpu(), lse.cpu(), o, m, z, BF)


# --------------------------------------------------------------------------- decode with weights
@pytest.mark.parametrize("lens,hq,hkv,d,dtype,bs,alibi,split,prev", [
    ([1], 1, 1, 8, FP, 16, False, 0, "none"),
    ([0, 17, 300, 1000], 8, 2, 64, BF, 16, True, 64, "other"),
    ([700, 40, 64], 6, 2, 80, FP, 32, False, 0, "same"),
    ([2000, 129], 12, 1, 128, BF, 16, True, 128, "none"),
    ([900, 1500], 8, 4, 256, BF, 64, False, 0, "other"),
    ([1300, 192], 160, 2, 64, FP, 192, False, 0, "same"),
])
def test_decode_weights(lens, hq, hkv, d, dtype, bs, alibi, split, prev):
    c = ref.Cache(lens, hq, hkv, d, dtype, bs, 51)
    n = len(lens)
    q, slopes = randn((n, hq, d), 52, dtype), slopes_of(hq, alibi)
    width = c.max + 5
    before = randn((n, hkv, width), 53, torch.float32)
    old = randn((n, hkv, width), 54, torch.float32).abs() if prev == "other" else None
    w = before.cuda().clone()
    kc, vc, table, cu = c.gpu()
    out, lse, got = mea.decode_paged_weights(
        q.cuda(), kc, vc, table, cu, c.max, w,
        prev_weights=w if prev == "same" else gpu(old), alibi_slopes=gpu(slopes), scale=d ** -0.5,
        split_keys=split)
    assert got is w
    o, m, z, want = ref.decode(c, q, d ** -0.5, slopes)
    ref.check_out(out.cpu(), lse.cpu(), o, m, z, dtype)
    got = got.cpu()
    base = {"none": torch.zeros_like(before), "other": old, "same": before}[prev]
    for b, length in enumerate(lens):
        want[b] = torch.stack(want[b])
        e = (got[b, :, :length].double() - want[b] - base[b, :, :length].double()).abs()
        bound = ref.F32 * want[b] + 2.0 ** -23 * (base[b, :, :length].abs() + want[b]) * (hq // hkv)
        assert bool((e <= bound + 1e-30).all()), float((e / (bound + 1e-30)).max())
        assert torch.equal(got[b, :, length:], before[b, :, length:])
    assert mea.device_error() == 0


# ------------------------------------------------------------------------------- prompt's weights
@pytest.mark.parametrize("lens_q,lens_k,hq,hkv,d,dtype,causal,alibi,last", [
    ([1], [1], 1, 1, 8, FP, True, False, 0),
    ([37, 120, 8, 200], [37, 120, 8, 200], 8, 8, 64, FP, True, False, 0),
    ([300, 0, 129], [300, 0, 129], 8, 2, 128, BF, True, True, 0),
    ([100, 5], [228, 300], 6, 2, 80, FP, True, True, 0),       # queries at the end of the keys
    ([130, 7], [40, 3], 4, 2, 128, BF, True, False, 0),         # first queries see no key
    ([257, 64], [100, 400], 12, 1, 128, BF, False, True, 0),
    ([257, 3], [129, 128], 4, 4, 40, FP, False, False, 0),
    ([700, 31, 32], [700, 31, 32], 8, 2, 128, BF, True, True, 32),
    ([700, 500], [700, 500], 8, 4, 256, BF, True, False, 129),
    ([300, 0], [300, 60], 4, 1, 256, FP, False, False, 1),
    ([260], [260], 6, 2, 136, BF, True, False, 0),
    ([300, 700], [300, 700], 64, 1, 64, BF, True, True, 3),  # 64 heads in a tile
])
def test_prompt_weights(lens_q, lens_k, hq, hkv, d, dtype, causal, alibi, last):
    q, k, v = make_qkv(lens_q, lens_k, hq, hkv, d, dtype, 61)
    slopes = slopes_of(hq, alibi)
    cq, ck = cu_seqlens(lens_q), cu_seqlens(lens_k)
    _, lse = mea.attention_packed(q.cuda(), k.cuda(), v.cuda(), cq.cuda(), ck.cuda(), max(lens_q),
                                  causal=causal, alibi_slopes=gpu(slopes), scale=d ** -0.5)
    width = max(lens_k) + 3
    before = randn((len(lens_q), hkv, width), 62, torch.float32)
    w = before.cuda().clone()
    got = mea.attention_packed_weights(q.cuda(), k.cuda(), lse, cq.cuda(), ck.cuda(), max(lens_q),
                                       max(lens_k), causal=causal, alibi_slopes=gpu(slopes),
                                       scale=d ** -0.5, last_queries=last, weights=w).cpu()
    want = ref.prompt_weights(q, k, lse.cpu(), lens_q, lens_k, d ** -0.5, causal, slopes, last,
                              width)
    for s, lk in enumerate(lens_k):
        e = (got[s, :, :lk].double() - want[s, :, :lk]).abs()
        bound = ref.F32 * want[s, :, :lk] + 1e-30
        assert bool((e <= bound).all()), float((e / bound).max())
        assert torch.equal(got[s, :, lk:], before[s, :, lk:])
    assert mea.device_error() == 0


def test_prompt_weights_ignore_a_neighbour_segment():
    """A segment's tile reaches into its neighbour's rows: NaN and infinities there change nothing."""
    lens = [70, 100]
    q, k, v = make_qkv(lens, lens, 2, 1, 64, BF, 63)
    cu = cu_seqlens(lens).cuda()
    _, lse = mea.attention_packed(q.cuda(), k.cuda(), v.cuda(), cu, cu, 100, causal=True)

    def run(q, k, lse):
        return mea.attention_packed_weights(q, k, lse, cu, cu, 100, 100, causal=True).cpu()[0]

    clean = run(q.cuda(), k.cuda(), lse)
    q[70:], k[70:] = math.inf, math.nan
    lse = lse.clone()
    lse[:, 70:] = math.nan
    assert torch.equal(run(q.cuda(), k.cuda(), lse), clean)


# -------------------------------------------------------------------------------------- eviction
@pytest.mark.parametrize("lens,hkv,d,dtype,bs,keep,recent,same", [
    ([1], 1, 8, FP, 16, 1, 0, False),
    ([0, 17, 300, 1000], 2, 64, BF, 16, 64, 10, False),
    ([700, 40], 2, 80, FP, 32, 100, 0, True),
    ([2000, 129], 1, 128, BF, 16, 128, 128, False),
    ([900, 1500], 4, 256, BF, 64, 500, 33, True),
    ([1300, 192], 3, 136, FP, 192, 191, 1, False),
    ([70000], 1, 16, FP, 64, 3000, 5, False),   # more keys than shared memory holds
])
def test_evict(lens, hkv, d, dtype, bs, keep, recent, same):
    n, per = len(lens), -(-min(keep, max(lens)) // bs)
    c = ref.Cache(lens, hkv, hkv, d, dtype, bs, 71, extra=n * per if same else 2)
    # Few distinct weights: ties everywhere.
    w = torch.randint(0, 9, (n, hkv, c.max + 2), generator=torch.Generator().manual_seed(72)).float()
    kc, vc, table, cu = c.gpu()
    if same:
        ids = torch.tensor(c.spare[:n * per], dtype=torch.int32).view(n, per)
        ko, vo, before = kc, vc, c.kc.clone()
    else:
        ids = torch.randperm(n * per, generator=torch.Generator().manual_seed(73)).to(torch.int32)
        ids = ids.view(n, per)
        before = randn((n * per, bs, hkv, d), 74, dtype)
        ko, vo = before.cuda().clone(), before.cuda().clone()
    kept, ow, ocu = mea.evict_paged(kc, vc, table, cu, c.max, w.cuda(), keep, recent, ids.cuda(),
                                    out_k_cache=None if same else ko,
                                    out_v_cache=None if same else vo)
    kept, ow, ko, vo = kept.cpu(), ow.cpu(), ko.cpu(), vo.cpu()
    left = [min(x, keep) for x in lens]
    assert ocu.cpu().tolist() == cu_seqlens(left).tolist()
    written = torch.zeros(before.shape[:3], dtype=torch.bool)
    for b, length in enumerate(lens):
        for g in range(hkv):
            m = max(0, length - recent)
            order = sorted(range(m), key=lambda t: (-float(w[b, g, t]), t))
            want = sorted(order[:max(0, left[b] - min(recent, length))]) + list(range(m, length))
            assert kept[b, g].tolist() == want + [-1] * (keep - len(want))
            assert torch.equal(ow[b, g], torch.cat((w[b, g, want], torch.zeros(keep - len(want)))))
            t = torch.arange(len(want))
            blk = ids[b, t // bs].long()
            assert torch.equal(ko[blk, t % bs, g], c.k[b][want, g])
            assert torch.equal(vo[blk, t % bs, g], c.v[b][want, g])
            written[blk, t % bs, g] = True
    # Nothing else was touched.
    assert torch.equal(ko[~written].nan_to_num(7.0), before[~written].nan_to_num(7.0))


@pytest.mark.parametrize("kind", ["spread", "close", "equal", "ties at the cut"])
@pytest.mark.parametrize("lens,hkv,keep,recent", [
    ([3001], 2, 700, 40),
    ([int(9 + 61 * i % 1300) for i in range(40)], 4, 150, 9),   # more (request, head)s than SMs
    ([60001], 1, 2000, 7),                                      # more keys than shared memory holds
])
def test_evict_selects_whatever_the_weights_range(lens, hkv, keep, recent, kind):
    n, bs = len(lens), 32
    c = ref.Cache(lens, hkv, hkv, 8, BF, bs, 76)
    w = randn((n, hkv, c.max), 77, torch.float32)
    if kind == "spread":
        w = torch.exp(12 * w)  # some 100 binades
    elif kind == "close":
        w = 1 + w.abs() * 2.0 ** -18
    elif kind == "equal":
        w = torch.full_like(w, 0.125)
    else:
        w = torch.where(w > 0.5, w, torch.full_like(w, 0.25))
    per = -(-keep // bs)
    ids = torch.arange(n * per, dtype=torch.int32).view(n, per)
    kc, vc, table, cu = c.gpu()
    ko = torch.zeros((n * per, bs, hkv, 8), dtype=BF, device="cuda")
    kept, ow, _ = mea.evict_paged(kc, vc, table, cu, c.max, w.cuda(), keep, recent, ids.cuda(),
                                  out_k_cache=ko, out_v_cache=torch.zeros_like(ko))
    kept, ow, ko = kept.cpu(), ow.cpu(), ko.cpu()
    for b, length in enumerate(lens):
        m = max(0, length - recent)
        for g in range(hkv):
            order = torch.sort(w[b, g, :m], descending=True, stable=True).indices.tolist()
            want = sorted(order[:max(0, min(length, keep) - min(recent, length))])
            want += list(range(m, length))
            assert kept[b, g].tolist() == want + [-1] * (keep - len(want))
            assert torch.equal(ow[b, g, :len(want)], w[b, g, want])
            t = torch.arange(len(want))
            assert torch.equal(ko[ids[b, t // bs].long(), t % bs, g], c.k[b][want, g])


def test_evict_ranks_nan_and_infinities():
    c = ref.Cache([10], 1, 1, 16, BF, 16, 75)
    kc, vc, table, cu = c.gpu()
    w = torch.tensor([[[0., -math.inf, 3., math.nan, math.inf, -0., 0., -5., 2., 9.]]])
    out = torch.zeros((1, 16, 1, 16), dtype=BF, device="cuda")
    table1 = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    kept, ow, _ = mea.evict_paged(kc, vc, table, cu, 10, w.cuda(), 6, 1, table1, out_k_cache=out,
                                  out_v_cache=out.clone())
    assert kept.cpu()[0, 0].tolist() == [0, 2, 3, 4, 8, 9]
    kept, _, _ = mea.evict_paged(kc, vc, table, cu, 10, w.cuda(), 8, 1, table1, out_k_cache=out,
                                 out_v_cache=out.clone())
    assert kept.cpu()[0, 0].tolist() == [0, 2, 3, 4, 5, 6, 8, 9]  # 0 and -0 are equal


# ------------------------------------------------------------------------------------------ tree
def random_tree(n, gen):
    return [int(torch.randint(-1, i, (1,), generator=gen)) if i else -1 for i in range(n)]


@pytest.mark.parametrize("lens,nq,hq,hkv,d,dtype,bs,alibi", [
    ([1], [1], 1, 1, 8, FP, 16, False),
    ([777], [8], 8, 8, 64, FP, 16, False),
    ([300, 40, 0, 129], [7, 40, 0, 1], 8, 2, 128, BF, 16, True),
    ([700, 128, 127], [33, 64, 1], 6, 2, 80, FP, 32, False),     # three heads a group
    ([2000, 129], [65, 100], 12, 1, 128, BF, 64, True),          # many row parts
    ([900, 1500, 3], [20, 5, 3], 8, 4, 256, BF, 128, False),
    ([385, 191], [12, 30], 4, 1, 256, FP, 192, True),
    ([5000], [17], 64, 8, 128, BF, 16, False),                   # one request over many CTAs
    ([256] * 70, [4] * 70, 8, 2, 40, FP, 64, True),
    ([3000, 1700, 129, 128], [16, 2, 1, 16], 16, 2, 128, BF, 16, True),  # one sub-tile's rows
    ([4000, 300] * 30, [40, 3] * 30, 16, 2, 64, FP, 32, False),  # one and two sub-tiles in turn
    ([500, 64], [11, 2], 4, 2, 136, BF, 32, False),              # a head dim that ends in a box
])
def test_tree(lens, nq, hq, hkv, d, dtype, bs, alibi):
    c = ref.Cache(lens, hq, hkv, d, dtype, bs, 81)
    gen = torch.Generator().manual_seed(82)
    parents = [random_tree(n, gen) for n in nq]
    mask = mea.tree_mask(parents)
    masks = []
    for t in parents:
        m = torch.eye(len(t), dtype=torch.bool)
        for i, p in enumerate(t):
            if p >= 0:
                m[i] |= m[p]
        masks.append(m)
    q, slopes = randn((sum(nq), hq, d), 83, dtype), slopes_of(hq, alibi)
    kc, vc, table, cu = c.gpu()
    out, lse = mea.decode_tree_paged(q.cuda(), kc, vc, table, cu_seqlens(nq).cuda(), cu, max(nq),
                                     c.max, mask.cuda(), alibi_slopes=gpu(slopes), scale=d ** -0.5)
    torch.cuda.synchronize()
    assert mea.device_error() == 0
    o, m, z = ref.tree(c, q, nq, masks, d ** -0.5, slopes)
    ref.check_out(out.cpu(), lse.cpu(), o, m, z, dtype)


@pytest.mark.parametrize("alibi", [False, True])
def test_tree_arbitrary_masks_and_empty_rows(alibi):
    """Masks that are no tree, rows that see nothing, set bits past the drafted tokens."""
    lens, nq, hq, hkv, d = [20, 70, 300], [20, 70, 40], 4, 2, 64
    c = ref.Cache(lens, hq, hkv, d, FP, 16, 84)
    gen = torch.Generator().manual_seed(85)
    masks = [torch.rand(n, n, generator=gen) < 0.4 for n in nq]
    masks[0][3] = masks[0][19] = masks[1][0] = False
    mask = torch.zeros((sum(nq), 4), dtype=torch.int64)
    row = 0
    for m in masks:
        for i in range(m.shape[0]):
            bits = sum(1 << j for j in range(m.shape[1]) if m[i, j]) | (((1 << 128) - 1) ^
                                                                       ((1 << m.shape[1]) - 1))
            for w in range(4):
                x = (bits >> (32 * w)) & 0xFFFFFFFF
                mask[row, w] = x - (1 << 32) if x >> 31 else x
            row += 1
    q, slopes = randn((sum(nq), hq, d), 86, FP), slopes_of(hq, alibi)
    kc, vc, table, cu = c.gpu()
    out, lse = mea.decode_tree_paged(q.cuda(), kc, vc, table, cu_seqlens(nq).cuda(), cu, 70, 300,
                                     mask.to(torch.int32).cuda(), alibi_slopes=gpu(slopes),
                                     scale=0.125)
    o, m, z = ref.tree(c, q, nq, masks, 0.125, slopes)
    assert int(torch.isinf(z).sum()) == 3 * hq
    ref.check_out(out.cpu(), lse.cpu(), o, m, z, FP)


def test_tree_of_a_chain_is_the_causal_forward():
    lens, nq = [200, 90], [33, 90]
    c = ref.Cache(lens, 8, 2, 128, BF, 32, 87)
    q = randn((sum(nq), 8, 128), 88, BF).cuda()
    kc, vc, table, cu = c.gpu()
    mask = mea.tree_mask([list(range(-1, n - 1)) for n in nq], device="cuda")
    sl = alibi_slope_values(8).cuda()
    cq = cu_seqlens(nq).cuda()
    out, lse = mea.decode_tree_paged(q, kc, vc, table, cq, cu, max(nq), 200, mask,
                                     alibi_slopes=sl, scale=0.09)
    k, v = torch.cat(c.k).cuda(), torch.cat(c.v).cuda()
    want, wl = mea.attention_packed(q, k, v, cq, cu, max(nq), causal=True, alibi_slopes=sl,
                                    scale=0.09)
    # Both within half a step of P and half a step of the result of the same values (of size <= 5).
    assert float((out.float() - want.float()).abs().max()) <= 2 * 2 * 2.0 ** -8 * 5
    assert float((lse - wl).abs().max()) <= 2 * ref.F32
