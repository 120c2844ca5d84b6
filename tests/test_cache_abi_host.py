"""Refusals of the paged-cache operators and of the prompt's attention weights, on the host: the
library's statuses (nothing is launched; no GPU is needed), the same calls through mea_call, and the
binding's checks of its tensors."""
import struct

import pytest
import torch

import memory_efficient_attention_b200 as mea
from memory_efficient_attention_b200 import _lib
from memory_efficient_attention_b200.build import build_library

A = 0x10000  # an aligned dummy address: never dereferenced, validation fails first

CALLS = {
    "mea_block_key_bounds": dict(k=A, table=A, cu=A, first=0, bounds=A, n=2, nb=10, bs=16, mb=5,
                                 max_k=70, hkv=8, d=128, dtype=1, stream=0),
    "mea_select_blocks": dict(q=A, bounds=A, table=A, cu=A, sel=A, n=2, nb=10, bs=16, mb=5,
                              max_k=70, hq=64, hkv=8, d=128, n_select=3, n_first=1, n_last=1,
                              dtype=1, stream=0),
    "mea_decode_selected": dict(q=A, k=A, v=A, table=A, cu=A, sel=A, out=A, lse=A, n=2, nb=10,
                                bs=16, mb=5, n_select=3, hq=64, hkv=8, d=128, scale=0.1, slopes=0,
                                dtype=1, ws=A, ws_bytes=1 << 30, stream=0),
    "mea_decode_weights": dict(q=A, k=A, v=A, table=A, cu=A, out=A, lse=A, weights=A, prev=0,
                               stride=70, n=2, nb=10, bs=16, mb=5, total_k=160, max_k=70, hq=64,
                               hkv=8, d=128, scale=0.1, slopes=0, dtype=1, ws=A,
                               ws_bytes=1 << 30, split=0, stream=0),
    "mea_attention_weights": dict(q=A, k=A, lse=A, cu_q=A, cu_k=A, weights=A, stride=70, n=2,
                                  total_q=100, total_k=120, max_q=60, max_k=70, hq=8, hkv=2,
                                  d=128, scale=0.1, mask=1, slopes=0, last=0, dtype=1, ws=A,
                                  ws_bytes=1 << 30, stream=0),
    "mea_evict_paged": dict(k=A, v=A, table=A, cu=A, weights=A, stride=70, ko=A, vo=A, ot=A,
                            kept=A, ow=A, ocu=A, n=2, nb=10, nob=10, bs=16, mb=5, mob=3, max_k=70,
                            hkv=8, d=128, n_keep=40, n_recent=8, dtype=1, stream=0),
    "mea_decode_tree": dict(q=A, k=A, v=A, table=A, cu_q=A, cu_k=A, mask=A, out=A, lse=A, n=2,
                            total_q=20, max_q=12, max_k=70, words=1, nb=10, bs=16, mb=5, hq=64,
                            hkv=8, d=128, scale=0.1, slopes=0, dtype=1, ws=A, ws_bytes=1 << 30,
                            stream=0),
}

N, S, H, D, T, L, C, W = (_lib.MEA_ERR_NULL, _lib.MEA_ERR_SHAPE, _lib.MEA_ERR_HEADS,
                          _lib.MEA_ERR_HEAD_DIM, _lib.MEA_ERR_DTYPE, _lib.MEA_ERR_ALIGN,
                          _lib.MEA_ERR_SCALE, _lib.MEA_ERR_WORKSPACE)
CASES = [
    ("mea_block_key_bounds", [
        (dict(k=0), N), (dict(bounds=0), N), (dict(n=0), S), (dict(n=70000), S), (dict(nb=0), S),
        (dict(bs=24), S), (dict(bs=96), S), (dict(mb=4), S), (dict(max_k=-1), S), (dict(hkv=0), H),
        (dict(d=12), D), (dict(d=264), D), (dict(dtype=2), T), (dict(bounds=A + 8), L),
        (dict(first=A + 2), L)]),
    ("mea_select_blocks", [
        (dict(q=0), N), (dict(sel=0), N), (dict(n=0), S), (dict(n_select=0), S),
        (dict(n_first=-1), S), (dict(n_last=-1), S), (dict(mb=4), S), (dict(bs=8), S),
        (dict(max_k=16 * 50001, mb=60000), S), (dict(hq=12), H), (dict(d=260), D),
        (dict(dtype=-1), T), (dict(q=A + 4), L), (dict(sel=A + 1), L)]),
    ("mea_decode_selected", [
        (dict(sel=0), N), (dict(out=0), N), (dict(n=0), S), (dict(n_select=0), S),
        (dict(n_select=1 << 27), S), (dict(bs=40), S), (dict(hkv=0), H), (dict(hq=20), H),
        (dict(d=4), D), (dict(dtype=9), T), (dict(scale=float("inf")), C), (dict(k=A + 8), L),
        (dict(sel=A + 2), L), (dict(ws=0), W), (dict(ws=A + 128), W)]),
    ("mea_decode_weights", [
        (dict(weights=0), N), (dict(k=0), N), (dict(stride=69), S), (dict(max_k=161), S),
        (dict(mb=4), S), (dict(split=65), S), (dict(split=-64), S), (dict(n=70000), S),
        (dict(hq=60), H), (dict(d=130), D), (dict(dtype=3), T), (dict(scale=float("nan")), C),
        (dict(weights=A + 2), L), (dict(prev=A + 1), L), (dict(ws=0), W), (dict(ws=A + 16), W)]),
    ("mea_attention_weights", [
        (dict(lse=0), N), (dict(weights=0), N), (dict(q=0), N), (dict(cu_q=0), N),
        (dict(stride=69), S), (dict(max_q=101), S), (dict(max_k=121), S), (dict(last=-1), S),
        (dict(n=0), S), (dict(hq=7), H), (dict(d=20), D), (dict(d=272), D), (dict(dtype=2), T),
        (dict(mask=2), _lib.MEA_ERR_MASK), (dict(scale=float("inf")), C), (dict(lse=A + 2), L),
        (dict(q=A + 8), L), (dict(ws=0), W), (dict(ws=A + 4), W)]),
    ("mea_evict_paged", [
        (dict(kept=0), N), (dict(ot=0), N), (dict(ocu=0), N), (dict(n_keep=0), S),
        (dict(n_recent=41), S), (dict(n_recent=-1), S), (dict(mob=2), S), (dict(nob=0), S),
        (dict(stride=60), S), (dict(mb=4), S), (dict(bs=17), S), (dict(hkv=0), H), (dict(d=0), D),
        (dict(dtype=2), T), (dict(ko=A + 8), L), (dict(kept=A + 2), L)]),
    ("mea_decode_tree", [
        (dict(mask=0), N), (dict(cu_q=0), N), (dict(max_q=21), S), (dict(words=0), S),
        (dict(max_q=20, total_q=40, words=0), S), (dict(max_q=33, total_q=40), S),
        (dict(mb=4), S), (dict(bs=48), S), (dict(n=0), S), (dict(total_q=1 << 30, max_q=30), S),
        (dict(hq=12), H), (dict(d=300), D), (dict(dtype=2), T), (dict(scale=float("nan")), C),
        (dict(out=A + 4), L), (dict(mask=A + 2), L), (dict(ws=0), W), (dict(ws=A + 64), W)]),
]


@pytest.fixture(scope="module")
def lib():
    build_library()
    return _lib.load()


@pytest.mark.parametrize("name,kw,rc", [(n, kw, rc) for n, rows in CASES for kw, rc in rows])
def test_refusals(lib, name, kw, rc):
    args = dict(CALLS[name])
    args.update(kw)
    values = [args[k] for k in args]
    assert getattr(lib, name)(*values) == rc
    entry, words = _lib.CALLS[name]
    assert lib.mea_call(entry, words.pack(*values)) == rc


def test_call_refuses_unknown_entries_and_sizes_past_an_int(lib):
    assert lib.mea_call(0, struct.pack("q", 0)) == S
    assert lib.mea_call(8, struct.pack("q", 0)) == S
    assert lib.mea_call(1, None) == N
    args = dict(CALLS["mea_block_key_bounds"], max_k=(1 << 32) + 5)
    entry, words = _lib.CALLS["mea_block_key_bounds"]
    assert lib.mea_call(entry, words.pack(*args.values())) == S


def test_workspace_sizes(lib):
    # Partial ranges: two per SM (148 on a host without a GPU).
    assert lib.mea_decode_tree_workspace_size(64, 8, 128) >= 2 * 148 * 256 * (128 + 1) * 4
    assert lib.mea_decode_tree_workspace_size(64, 8, 256) >= 2 * 148 * 128 * (256 + 1) * 4
    assert lib.mea_decode_tree_workspace_size(64, 7, 128) == 0
    assert lib.mea_decode_selected_workspace_size(4, 64, 16, 64, 8, 128) >= 2 * 148 * 8 * 129 * 4
    assert lib.mea_decode_selected_workspace_size(4, 64, 24, 64, 8, 128) == 0
    assert lib.mea_attention_weights_workspace_size(128) >= 2 * 148 * 256 * 4
    assert lib.mea_attention_weights_workspace_size(3) == 0
    base = lib.mea_decode_workspace_size(4, 1000, 16, 4, 128, 256)
    slots = -(-1000 // 256) + 4
    assert lib.mea_decode_weights_workspace_size(4, 1000, 16, 4, 128, 256) == \
        base + slots * 16 * 256 * 4
    assert lib.mea_decode_weights_workspace_size(0, 1000, 16, 4, 128, 256) == 0


# ---------------------------------------------------------------------------------- the binding
def test_binding_refuses_host_tensors():
    kc = torch.zeros((4, 16, 2, 64), dtype=torch.float16)
    q = torch.zeros((2, 8, 64), dtype=torch.float16)
    table = torch.zeros((2, 2), dtype=torch.int32)
    cu = torch.tensor([0, 4, 20], dtype=torch.int32)
    w = torch.zeros((2, 2, 20))
    sel = torch.zeros((2, 2, 1), dtype=torch.int32)
    b = torch.zeros((4, 2, 2, 64), dtype=torch.float16)
    for call in (lambda: mea.block_key_bounds(kc, table, cu, 16),
                 lambda: mea.select_blocks(q, b, table, cu, 16, 16, 1),
                 lambda: mea.decode_paged_selected(q, kc, kc, table, cu, sel),
                 lambda: mea.decode_paged_weights(q, kc, kc, table, cu, 16, w),
                 lambda: mea.attention_packed_weights(q, q, torch.zeros(8, 2), cu, cu, 1, 1),
                 lambda: mea.evict_paged(kc, kc, table, cu, 16, w, 8, 0, table),
                 lambda: mea.decode_tree_paged(q, kc, kc, table, cu, cu, 1, 16,
                                               torch.ones((2, 1), dtype=torch.int32))):
        with pytest.raises(mea.MeaError) as e:
            call()
        assert e.value.rc == _lib.MEA_ERR_DEVICE


def test_tree_mask():
    m = mea.tree_mask([[-1, 0, 0, 2], [], [-1]])
    assert m.dtype == torch.int32 and m.flatten().tolist() == [1, 3, 5, 13, 1]
    long = mea.tree_mask([list(range(-1, 69))])
    assert tuple(long.shape) == (70, 3)
    assert long[31].tolist() == [-1, 0, 0] and long[69].tolist() == [-1, -1, 63]
    assert tuple(mea.tree_mask([]).shape) == (0, 1)
    for bad in ([0], [-1, 1], [-1, -2]):
        with pytest.raises(ValueError):
            mea.tree_mask([bad])
