"""Outputs of the cache operators that overlap what the same call reads are refused, on the host
(nothing is launched; no GPU is needed)."""
import pytest

from memory_efficient_attention_b200 import _lib
from memory_efficient_attention_b200.build import build_library

S, MB = _lib.MEA_ERR_SHAPE, 1 << 20
# Dummy addresses a megabyte apart: never dereferenced, the library has no GPU here or refuses first.
EVICT = {name: (i + 1) * MB for i, name in enumerate(
    ("k", "v", "table", "cu", "weights", "stride", "ko", "vo", "ot", "kept", "ow", "ocu"))}
EVICT.update(stride=70, n=2, nb=10, nob=10, bs=16, mb=5, mob=3, max_k=70, hkv=8, d=128, n_keep=40,
             n_recent=8, dtype=1, stream=0)


@pytest.fixture(scope="module")
def lib():
    build_library()
    return _lib.load()


def both(lib, name, args):
    entry, words = _lib.CALLS[name]
    rc = getattr(lib, name)(*args.values())
    assert lib.mea_call(entry, words.pack(*args.values())) == rc
    return rc


W_BYTES, KEPT_BYTES = 2 * 8 * 70 * 4, 2 * 8 * 40 * 4


@pytest.mark.parametrize("out,at", [
    ("ocu", EVICT["cu"]),                       # lengths updated in place
    ("ocu", EVICT["cu"] + 2 * 4), ("ocu", EVICT["cu"] - 2 * 4),
    ("ow", EVICT["weights"]),                   # weights updated in place
    ("ow", EVICT["weights"] + W_BYTES - 4), ("ow", EVICT["weights"] - KEPT_BYTES + 4),
    ("kept", EVICT["table"]), ("kept", EVICT["ot"] + 4), ("ocu", EVICT["ot"]),
    ("kept", EVICT["ow"]), ("ocu", EVICT["kept"] + KEPT_BYTES - 4),
])
def test_eviction_refuses_updates_in_place(lib, out, at):
    assert both(lib, "mea_evict_paged", dict(EVICT, **{out: at})) == S


WEIGHTS = {name: (i + 1) * MB for i, name in enumerate(
    ("q", "k", "v", "table", "cu", "out", "lse", "weights", "prev"))}
WEIGHTS.update(stride=70, n=2, nb=10, bs=16, mb=5, total_k=160, max_k=70, hq=64, hkv=8, d=128,
               scale=0.1, slopes=0, dtype=1, ws=MB * 16, ws_bytes=1 << 30, split=0, stream=0)


@pytest.mark.parametrize("shift", [4, -4, 70 * 4, W_BYTES - 4, 4 - W_BYTES])
def test_weights_refuse_a_shifted_previous_sum(lib, shift):
    """weights itself accumulates in place; a tensor that overlaps it in another way does not."""
    args = dict(WEIGHTS, prev=WEIGHTS["weights"] + shift)
    assert both(lib, "mea_decode_weights", args) == S


@pytest.mark.parametrize("out,at", [
    ("ow", EVICT["weights"] + W_BYTES), ("ow", EVICT["weights"] - KEPT_BYTES),
    ("ocu", EVICT["cu"] + 3 * 4), ("ocu", EVICT["cu"] - 3 * 4),
])
def test_neighbouring_buffers_do_not_overlap(lib, out, at):
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch on dummy addresses")
    rc = both(lib, "mea_evict_paged", dict(EVICT, **{out: at}))
    assert rc in (_lib.MEA_ERR_CUDA, _lib.MEA_ERR_DEVICE)  # past the checks: there is no GPU
    for prev in (0, WEIGHTS["weights"], WEIGHTS["weights"] + W_BYTES):
        rc = both(lib, "mea_decode_weights", dict(WEIGHTS, prev=prev))
        assert rc in (_lib.MEA_ERR_CUDA, _lib.MEA_ERR_DEVICE)
