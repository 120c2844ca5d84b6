"""The paged-cache operators as a serving program uses them: one after the other on one cache, in a
CUDA graph, on another stream, with strided queries, far into a large cache, and the binding's
refusals on the GPU."""
import math

import pytest
import torch

import cache_reference as ref
import memory_efficient_attention_b200 as mea
from memory_efficient_attention_b200 import _lib
from mea_workloads import alibi_slope_values, cu_seqlens, make_qkv, randn

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def test_prompt_then_evict_then_decode():
    """A prompt's attention weights decide what stays; the decode over the new cache is the softmax over
    the kept keys, whichever they are for each head."""
    lens, hq, hkv, d, bs, keep = [500, 130, 40], 8, 2, 128, 16, 100
    q, k, v = make_qkv(lens, lens, hq, hkv, d, BF, 5)
    cu = cu_seqlens(lens).cuda()
    _, lse = mea.attention_packed(q.cuda(), k.cuda(), v.cuda(), cu, cu, 500, causal=True)
    w = mea.attention_packed_weights(q.cuda(), k.cuda(), lse, cu, cu, 500, 500, causal=True,
                                     last_queries=64)
    c = ref.Cache(lens, hq, hkv, d, BF, bs, 5)
    c.k, c.v = list(torch.split(k, lens)), list(torch.split(v, lens))
    for b, n in enumerate(lens):
        for t in range(n):
            c.kc[c.table[b, t // bs], t % bs], c.vc[c.table[b, t // bs], t % bs] = \
                c.k[b][t], c.v[b][t]
    kc, vc, table, cuk = c.gpu()
    per = -(-keep // bs)
    ko = torch.full((3 * per, bs, hkv, d), math.nan, dtype=BF, device="cuda")
    vo = torch.full_like(ko, math.nan)
    ot = torch.arange(3 * per, dtype=torch.int32, device="cuda").view(3, per).flip(0).contiguous()
    kept, w2, cu2 = mea.evict_paged(kc, vc, table, cuk, 500, w, keep, 20, ot, out_k_cache=ko,
                                    out_v_cache=vo)
    kept = kept.cpu()
    keys = [[[t for t in kept[b, g].tolist() if t >= 0] for g in range(hkv)] for b in range(3)]
    assert [len(x[0]) for x in keys] == [100, 100, 40]
    assert cu2.cpu().tolist() == [0, 100, 200, 240]
    qd = randn((3, hq, d), 6, BF)
    # The next step attends to what is left and adds its weights.
    out, lse, w3 = mea.decode_paged_weights(qd.cuda(), ko, vo, ot, cu2, keep, w2, prev_weights=w2)
    o, m, z, dw = ref.decode(c, qd, d ** -0.5, None, keys)
    ref.check_out(out.cpu(), lse.cpu(), o, m, z, BF)
    w = w.cpu()
    for b in range(3):
        for g in range(hkv):
            old = w[b, g, keys[b][g]]
            got = w3[b, g, :len(old)].cpu().double()
            bound = ref.F32 * dw[b][g] + 2.0 ** -23 * (old.abs() + dw[b][g]) * (hq // hkv)
            assert bool(((got - old.double() - dw[b][g]).abs() <= bound + 1e-30).all())
    # The plain paged decode reads the new cache alike.
    out2, lse2 = mea.decode_paged(qd.cuda(), ko, vo, ot, cu2, keep)
    ref.check_out(out2.cpu(), lse2.cpu(), o, m, z, BF)
    assert mea.device_error() == 0


def test_choice_of_every_block_is_the_paged_decode():
    lens = [700, 33, 64]
    c = ref.Cache(lens, 16, 4, 64, FP, 32, 9)
    kc, vc, table, cu = c.gpu()
    q = randn((3, 16, 64), 10, FP).cuda()
    sl = alibi_slope_values(16).cuda()
    bounds = mea.block_key_bounds(kc, table, cu, 700)
    sel = mea.select_blocks(q, bounds, table, cu, 700, 32, 40)
    out, lse = mea.decode_paged_selected(q, kc, vc, table, cu, sel, alibi_slopes=sl)
    want, wl = mea.decode_paged(q, kc, vc, table, cu, 700, alibi_slopes=sl)
    # Both round P and the result once each, of values of size up to 5.
    assert float((out.float() - want.float()).abs().max()) <= 4 * 2.0 ** -11 * 5
    assert float((lse - wl).abs().max()) <= 2 * ref.F32


def _step(s):
    """One serving step through every operator; returns its outputs."""
    mea.block_key_bounds(s["kc"], s["table"], s["cu"], s["max"], first_key=s["first"],
                         bounds=s["bounds"])
    sel = mea.select_blocks(s["q"], s["bounds"], s["table"], s["cu"], s["max"], 16, 6,
                            selected=s["sel"])
    mea.decode_paged_selected(s["q"], s["kc"], s["vc"], s["table"], s["cu"], sel, scale=0.1,
                              workspace=s["ws"], out=s["o1"], lse=s["l1"])
    mea.decode_paged_weights(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["max"], s["w"],
                             scale=0.1, workspace=s["ws"], total_k_bound=s["total"], out=s["o2"],
                             lse=s["l2"])
    mea.decode_tree_paged(s["qt"], s["kc"], s["vc"], s["table"], s["cuq"], s["cu"], 9, s["max"],
                          s["mask"], alibi_slopes=s["sl"], scale=0.1, workspace=s["ws"],
                          out=s["o3"], lse=s["l3"])
    mea.attention_packed_weights(s["qt"], s["kp"], s["l3"], s["cuq"], s["cu"], 9, s["max"],
                                 causal=True, scale=0.1, weights=s["wp"], workspace=s["ws"])
    mea.evict_paged(s["kc"], s["vc"], s["table"], s["cu"], s["max"], s["w"], 50, 7, s["ot"],
                    out_k_cache=s["ko"], out_v_cache=s["vo"], kept=s["kept"], out_weights=s["w2"],
                    out_cu_seqlens_k=s["cu2"])
    return [s[k] for k in ("bounds", "sel", "o1", "l1", "o2", "l2", "w", "o3", "l3", "wp", "kept",
                           "w2", "cu2", "ko", "vo")]


def _state():
    lens, nq, hq, hkv, d, bs = [300, 9, 1000, 64], [9, 9, 4, 1], 8, 2, 128, 16
    c = ref.Cache(lens, hq, hkv, d, BF, bs, 15)
    kc, vc, table, cu = c.gpu()
    dev = dict(device="cuda")
    s = {"kc": kc, "vc": vc, "table": table, "cu": cu, "max": 1000, "total": sum(lens),
         "first": torch.tensor([290, 0, 0, 63], dtype=torch.int32, **dev),
         "bounds": torch.zeros((kc.shape[0], hkv, 2, d), dtype=BF, **dev),
         "sel": torch.empty((4, hkv, 6), dtype=torch.int32, **dev),
         "q": randn((4, hq, d), 16, BF, "cuda"), "qt": randn((23, hq, d), 17, BF, "cuda"),
         "kp": randn((sum(lens), hkv, d), 18, BF, "cuda"), "cuq": cu_seqlens(nq).cuda(),
         "mask": mea.tree_mask([[-1] + [0] * (n - 1) for n in nq], device="cuda"),
         "sl": alibi_slope_values(hq).cuda(), "w": torch.zeros((4, hkv, 1000), **dev),
         "wp": torch.zeros((4, hkv, 1000), **dev),
         "ot": torch.randperm(16, dtype=torch.int32, **dev).view(4, 4).contiguous(),
         "kept": torch.empty((4, hkv, 50), dtype=torch.int32, **dev),
         "w2": torch.empty((4, hkv, 50), **dev), "cu2": torch.empty(5, dtype=torch.int32, **dev)}
    s["ko"] = torch.zeros((16, bs, hkv, d), dtype=BF, **dev)
    s["vo"] = torch.zeros_like(s["ko"])
    for i, (rows, like) in enumerate((((4, "q"), (4, "q"), (23, "qt")))):
        s[f"o{i + 1}"] = torch.empty_like(s[like])
        s[f"l{i + 1}"] = torch.empty((hq, rows), **dev)
    n = max(mea.decode_weights_workspace_size(4, sum(lens), hq, hkv, d),
            mea.decode_selected_workspace_size(4, 6, bs, hq, hkv, d),
            mea.decode_tree_workspace_size(hq, hkv, d), mea.attention_weights_workspace_size(d))
    s["ws"] = torch.empty(n, dtype=torch.uint8, **dev)
    return s


def test_a_step_replays_in_a_cuda_graph_and_on_another_stream():
    """Every operator in one graph: bit for bit the eager results, again after the inputs changed, and
    the same on a side stream. (No atomics anywhere: all of it is deterministic.)"""
    s = _state()
    fixed = [t.clone() for t in _step(s)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a, b in zip(fixed, _step(s)):
            assert torch.equal(a, b)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            outs = _step(s)
    torch.cuda.synchronize()
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(fixed, outs):
        assert torch.equal(a, b)
    s["q"].copy_(randn(tuple(s["q"].shape), 21, BF, "cuda"))
    s["qt"].copy_(randn(tuple(s["qt"].shape), 22, BF, "cuda"))
    s["kc"][s["table"][0, 18]] = 2.0  # the block of the first request's last keys
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in outs]
    for a, b in zip(got, _step(s)):
        assert torch.equal(a, b)
    assert not torch.equal(got[7], fixed[7])
    assert mea.device_error() == 0


@pytest.mark.parametrize("split", [0, 64])
def test_requests_that_share_their_first_blocks(split):
    """Three requests with one prefix: together they have more keys than the cache has slots."""
    length, hq, hkv, d, bs, dtype = 1200, 8, 2, 64, 16, BF
    c = ref.Cache([length], hq, hkv, d, dtype, bs, 91, extra=8)
    c.lens = [1200, 1200, 960]
    c.k, c.v = [c.k[0][:n] for n in c.lens], [c.v[0][:n] for n in c.lens]
    c.table, c.cu = c.table.expand(3, -1).contiguous(), cu_seqlens(c.lens)
    assert sum(c.lens) > c.num_blocks * bs
    q = randn((3, hq, d), 92, dtype)
    kc, vc, table, cu = c.gpu()
    w = torch.zeros((3, hkv, length), device="cuda")
    out, lse, _ = mea.decode_paged_weights(q.cuda(), kc, vc, table, cu, length, w, scale=0.125,
                                           split_keys=split)
    o, m, z, want = ref.decode(c, q, 0.125)
    ref.check_out(out.cpu(), lse.cpu(), o, m, z, dtype)
    for b, n in enumerate(c.lens):
        x = torch.stack(want[b])
        assert bool(((w.cpu()[b, :, :n].double() - x).abs() <=
                     ref.F32 * x + 2.0 ** -23 * x * (hq // hkv) + 1e-30).all())
        assert not bool(w[b, :, n:].any())
    bounds = mea.block_key_bounds(kc, table, cu, length)
    full, used = ref.block_bounds(c)
    assert torch.equal(bounds.cpu()[used], full[used])
    sel = mea.select_blocks(q.cuda(), bounds, table, cu, length, bs, 9)
    assert sel.cpu().tolist() == ref.choose(c, q, full, 9, 1, 1)
    # Tokens drafted for all three: their keys lie in the shared blocks here.
    nq = [5, 3, 16]
    tq = randn((sum(nq), hq, d), 93, dtype)
    chain = [list(range(-1, n - 1)) for n in nq]
    got, gl = mea.decode_tree_paged(tq.cuda(), kc, vc, table, cu_seqlens(nq).cuda(), cu, 16, length,
                                    mea.tree_mask(chain).cuda(), scale=0.125)
    o, m, z = ref.tree(c, tq, nq, [torch.ones(n, n, dtype=torch.bool).tril() for n in nq], 0.125)
    ref.check_out(got.cpu(), gl.cpu(), o, m, z, dtype)


def test_rows_behind_the_last_request_stay():
    """Buffers longer than the batch, and bounds on the lengths that are too large, as a captured step
    has them: what lies behind the last request is neither read nor written."""
    lens, nq, hq, hkv, d, bs = [300, 0, 77], [5, 0, 33], 8, 2, 128, 16
    c = ref.Cache(lens, hq, hkv, d, BF, bs, 94)
    kc, vc, table, cu = c.gpu()
    table = torch.cat((table, torch.full((3, 100), 1 << 30, dtype=torch.int32, device="cuda")), 1)
    rows, tq = sum(nq), sum(nq) + 40
    q = randn((tq, hq, d), 95, BF)
    q[rows:] = math.nan
    chain = [list(range(-1, n - 1)) for n in nq]
    mask = torch.full((tq, 4), -1, dtype=torch.int32)
    mask[:rows, :2] = mea.tree_mask(chain)
    before = randn((tq, hq, d), 96, BF)
    lse0 = randn((hq, tq), 97, torch.float32)
    out, lse = before.cuda(), lse0.cuda()
    mea.decode_tree_paged(q.cuda(), kc, vc, table, cu_seqlens(nq).cuda(), cu, 78, 1800, mask.cuda(),
                          scale=0.09, out=out, lse=lse)
    o, m, z = ref.tree(c, q[:rows], nq, [torch.ones(n, n, dtype=torch.bool).tril() for n in nq],
                       0.09)
    ref.check_out(out.cpu()[:rows], lse.cpu()[:, :rows], o, m, z, BF)
    assert torch.equal(out.cpu()[rows:], before[rows:])
    assert torch.equal(lse.cpu()[:, rows:], lse0[:, rows:])
    # A packed prompt with rows of padding.
    pq, pk, pv = make_qkv(lens, lens, hq, hkv, d, BF, 98)
    cuq = cu_seqlens(lens).cuda()
    _, pl = mea.attention_packed(pq.cuda(), pk.cuda(), pv.cuda(), cuq, cuq, 300, causal=True)
    want = mea.attention_packed_weights(pq.cuda(), pk.cuda(), pl, cuq, cuq, 300, 300, causal=True)
    pad = torch.full((50, hq, d), math.nan, dtype=BF)
    w = torch.full((3, hkv, 400), 7.0, device="cuda")
    got = mea.attention_packed_weights(
        torch.cat((pq, pad)).cuda(), torch.cat((pk, pad[:, :hkv])).cuda(),
        torch.cat((pl, torch.full((hq, 50), math.nan, device="cuda")), 1).contiguous(), cuq, cuq,
        400, 400, causal=True, weights=w)
    for b, n in enumerate(lens):
        # (other bounds may cut the sums elsewhere: fp32 rounding)
        assert bool(((got[b, :, :n] - want[b, :, :n]).abs() <= ref.F32 * want[b, :, :n]).all())
        assert bool((got[b, :, n:] == 7.0).all())
    assert mea.device_error() == 0


def test_two_streams_at_once():
    """Two steps in flight together, each with its own buffers and workspace."""
    a, b = _state(), _state()
    b["q"].copy_(randn(tuple(b["q"].shape), 31, BF, "cuda"))
    want_a, want_b = [t.clone() for t in _step(a)], [t.clone() for t in _step(b)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            got_a = _step(a)
        with torch.cuda.stream(s2):
            got_b = _step(b)
    torch.cuda.synchronize()
    for x, y in zip(want_a + want_b, got_a + got_b):
        assert torch.equal(x, y)


def test_strided_queries_and_lists():
    """Queries, masks, lists and lengths that are views: read as what they hold."""
    s = _state()
    wide = torch.randn((4, 2, 8, 128), device="cuda").to(BF)
    q = wide[:, 1]
    assert not q.is_contiguous()
    sel = mea.select_blocks(q, s["bounds"], s["table"], s["cu"], 1000, 16, 6)
    assert torch.equal(sel, mea.select_blocks(q.contiguous(), s["bounds"], s["table"], s["cu"], 1000,
                                              16, 6))
    twice = sel.repeat_interleave(2, 2)[:, :, ::2]
    cu2 = s["cu"].repeat_interleave(2)[::2]
    table = torch.cat((s["table"], s["table"]), 1)[:, :s["table"].shape[1]]
    x = mea.decode_paged_selected(q, s["kc"], s["vc"], table, cu2, twice)
    y = mea.decode_paged_selected(q.contiguous(), s["kc"], s["vc"], s["table"], s["cu"], sel)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    mask = s["mask"].repeat(1, 2)[:, :1]
    qt = s["qt"].transpose(0, 1).contiguous().transpose(0, 1)
    x = mea.decode_tree_paged(qt, s["kc"], s["vc"], table, s["cuq"], cu2, 9, 1000, mask)
    y = mea.decode_tree_paged(s["qt"], s["kc"], s["vc"], s["table"], s["cuq"], s["cu"], 9, 1000,
                              s["mask"])
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_far_into_a_large_cache():
    """Blocks past 2^31 elements (and 2^32 bytes): the same results as in a small cache."""
    lens, hq, hkv, d, bs = [90, 200], 8, 2, 128, 64
    c = ref.Cache(lens, hq, hkv, d, BF, bs, 41)
    kc, vc, table, cu = c.gpu()
    nb = (1 << 31) // (bs * hkv * d) + 64
    big_k = torch.empty((nb, bs, hkv, d), dtype=BF, device="cuda")
    big_v = torch.empty_like(big_k)
    far = nb - kc.shape[0]
    big_k[far:], big_v[far:] = kc, vc
    live = torch.where(table >= kc.shape[0], table, table + far)
    q = randn((2, hq, d), 42, BF, "cuda")
    qt = randn((7, hq, d), 43, BF, "cuda")
    cuq, mask = cu_seqlens([3, 4]).cuda(), mea.tree_mask([[-1, 0, 0], [-1, 0, 1, 1]], device="cuda")
    w = torch.rand((2, hkv, 200), device="cuda")
    ot = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)

    def run(k, v, t):
        b = mea.block_key_bounds(k, t, cu, 200)
        sel = mea.select_blocks(q, b, t, cu, 200, bs, 2)
        o1, l1 = mea.decode_paged_selected(q, k, v, t, cu, sel)
        w1 = torch.zeros_like(w)
        o2, l2, _ = mea.decode_paged_weights(q, k, v, t, cu, 200, w1, total_k_bound=290)
        o3, l3 = mea.decode_tree_paged(qt, k, v, t, cuq, cu, 4, 200, mask)
        ko = torch.zeros((4, bs, hkv, d), dtype=BF, device="cuda")
        vo = torch.zeros_like(ko)
        kept, ow, _ = mea.evict_paged(k, v, t, cu, 200, w, 100, 5, ot, out_k_cache=ko,
                                      out_v_cache=vo)
        last = b[t[1, 3].long()].clone()
        # and out of a small cache into blocks far into the large one
        mea.evict_paged(kc, vc, table, cu, 200, w, 100, 5, ot + (nb - 4), out_k_cache=big_k2,
                        out_v_cache=big_v2)
        return [sel, o1, l1, o2, l2, w1, o3, l3, kept, ow, ko, vo, last, big_k2[nb - 4:].clone()]

    big_k2, big_v2 = torch.zeros_like(big_k), torch.zeros_like(big_v)
    for x, y in zip(run(kc, vc, table), run(big_k, big_v, live)):
        assert torch.equal(x, y)
    assert torch.equal(big_k2[nb - 4:], run(kc, vc, table)[10])


def test_tree_masked_keys_do_not_count():
    """NaN and infinite keys among drafted tokens that a row does not see leave that row alone."""
    lens, n, hq, hkv, d = [140], 12, 4, 2, 64
    c = ref.Cache(lens, hq, hkv, d, BF, 16, 51)
    kc, vc, table, cu = c.gpu()
    q = randn((n, hq, d), 52, BF, "cuda")
    parents = [-1, 0, 1, 0, 3, 4, -1, 6, 6, 8, 9, 10]
    mask, cuq = mea.tree_mask([parents], device="cuda"), cu_seqlens([n]).cuda()
    out, lse = mea.decode_tree_paged(q, kc, vc, table, cuq, cu, n, 140, mask)
    bad = 128 + 6  # token 6: seen by 6 to 11
    kc[table[0, bad // 16].long(), bad % 16] = math.nan
    out2, lse2 = mea.decode_tree_paged(q, kc, vc, table, cuq, cu, n, 140, mask)
    assert torch.equal(out[:6], out2[:6]) and torch.equal(lse[:, :6], lse2[:, :6])


def test_binding_refuses_what_does_not_match():
    s = _state()
    kc, vc, table, cu, q = s["kc"], s["vc"], s["table"], s["cu"], s["q"]
    S, T, D, W = (_lib.MEA_ERR_SHAPE, _lib.MEA_ERR_DTYPE, _lib.MEA_ERR_DEVICE,
                  _lib.MEA_ERR_WORKSPACE)
    calls = [
        (S, lambda: mea.decode_paged_selected(q[:, :, :64], kc, vc, table, cu, s["sel"])),
        (T, lambda: mea.decode_paged_selected(q.half(), kc, vc, table, cu, s["sel"])),
        (S, lambda: mea.decode_paged_selected(q, kc, vc, table, cu, s["sel"].long())),
        (S, lambda: mea.decode_paged_selected(q, kc, vc, table, cu[:4], s["sel"])),
        (S, lambda: mea.decode_paged_selected(q, kc.transpose(1, 2), vc, table, cu, s["sel"])),
        (S, lambda: mea.decode_paged_selected(q, kc, vc[1:], table, cu, s["sel"])),
        (D, lambda: mea.decode_paged_selected(q, kc, vc, table.cpu(), cu, s["sel"])),
        (D, lambda: mea.decode_paged_selected(q, kc, vc, table, cu, s["sel"].cpu())),
        (S, lambda: mea.decode_paged_selected(q, kc, vc, table, cu, s["sel"], out=q[:, :4])),
        (W, lambda: mea.decode_paged_selected(q, kc, vc, table, cu, s["sel"],
                                              workspace=s["ws"][:256])),
        (W, lambda: mea.decode_paged_selected(q, kc, vc, table, cu, s["sel"],
                                              workspace=s["ws"][8:])),
        (S, lambda: mea.select_blocks(q, s["bounds"], table, cu, 1000, 16, 0)),
        (S, lambda: mea.select_blocks(q, s["bounds"][:, :, :1], table, cu, 1000, 16, 4)),
        (S, lambda: mea.select_blocks(q[:2], s["bounds"], table, cu, 1000, 16, 4)),
        (S, lambda: mea.block_key_bounds(kc, table, cu, 10 ** 6)),
        (S, lambda: mea.block_key_bounds(kc, table, cu, 1000, first_key=s["first"][:2])),
        (S, lambda: mea.decode_paged_weights(q, kc, vc, table, cu, 1000, s["w"][:, :, :999])),
        (S, lambda: mea.decode_paged_weights(q, kc, vc, table, cu, 1000, s["w"].double())),
        (S, lambda: mea.decode_paged_weights(q, kc, vc, table, cu, 1000, s["w"],
                                             prev_weights=s["w"][:, :1])),
        (S, lambda: mea.decode_paged_weights(q, kc, vc, table, cu, 1000, s["w"],
                                             total_k_bound=500)),
        (S, lambda: mea.attention_packed_weights(s["qt"], s["kp"], s["l1"], s["cuq"], cu, 9, 1000)),
        (S, lambda: mea.attention_packed_weights(s["qt"], s["kp"], s["l3"], s["cuq"], cu[:3], 9,
                                                 1000)),
        (S, lambda: mea.attention_packed_weights(s["qt"], s["kp"], s["l3"], s["cuq"], cu, 9, 1000,
                                                 last_queries=-2)),
        (S, lambda: mea.evict_paged(kc, vc, table, cu, 1000, s["w"], 50, 51, s["ot"])),
        (S, lambda: mea.evict_paged(kc, vc, table, cu, 1000, s["w"], 100, 5, s["ot"])),
        (S, lambda: mea.evict_paged(kc, vc, table, cu, 1000, s["w"], 0, 0, s["ot"])),
        (S, lambda: mea.evict_paged(kc, vc, table, cu, 1000, s["w"], 50, 5, s["ot"],
                                    out_k_cache=s["ko"][:, :8], out_v_cache=s["vo"])),
        (S, lambda: mea.decode_tree_paged(s["qt"], kc, vc, table, s["cuq"], cu, 40, 1000,
                                          s["mask"])),
        (S, lambda: mea.decode_tree_paged(s["qt"], kc, vc, table, s["cuq"], cu, 9, 1000,
                                          s["mask"][:5])),
        (S, lambda: mea.decode_tree_paged(s["qt"], kc, vc, table, s["cuq"], cu, 9, 1000,
                                          s["mask"], alibi_slopes=s["sl"][:3])),
    ]
    for rc, call in calls:
        with pytest.raises(mea.MeaError) as e:
            call()
        assert e.value.rc == rc, call
    torch.cuda.synchronize()
    assert mea.device_error() == 0


def test_nothing_to_do():
    """Empty batches of tokens and requests without keys."""
    c = ref.Cache([0, 5], 4, 2, 64, FP, 16, 61)
    kc, vc, table, cu = c.gpu()
    q0 = torch.empty((0, 4, 64), dtype=FP, device="cuda")
    cu0 = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = mea.decode_tree_paged(q0, kc, vc, table, cu0, cu, 0, 5,
                                     torch.empty((0, 1), dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    k = torch.randn((5, 2, 64), device="cuda").half()
    w = mea.attention_packed_weights(q0, k, torch.empty((4, 0), device="cuda"), cu0, cu, 0, 5)
    assert bool((w == 0).all()) and w.shape == (2, 2, 5)
    q = torch.randn((2, 4, 64), device="cuda").half()
    none = torch.full((2, 2, 3), -1, dtype=torch.int32, device="cuda")
    out, lse = mea.decode_paged_selected(q, kc, vc, table, cu, none)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    w = torch.full((2, 2, 5), 7.0, device="cuda")
    out, lse, _ = mea.decode_paged_weights(q, kc, vc, table, cu, 5, w)
    assert bool((out[0] == 0).all()) and bool((lse[:, 0] == -math.inf).all())
    assert bool((w[0] == 7).all()) and bool(torch.isfinite(out[1]).all())
    assert mea.device_error() == 0
