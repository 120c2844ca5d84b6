"""Batches whose requests have no keys yet: weights of no entries (a null pointer) are no error."""
import pytest
import torch

import test_cache_abi_host as abi
from memory_efficient_attention_b200 import _lib

lib = abi.lib


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on dummy addresses")
@pytest.mark.parametrize("name,kw", [
    ("mea_decode_weights", dict(weights=0, stride=0, max_k=0, total_k=0)),
    ("mea_evict_paged", dict(weights=0, stride=0, max_k=0, cu=1 << 20, table=2 << 20, ot=3 << 20,
                             kept=4 << 20, ow=5 << 20, ocu=6 << 20)),
    ("mea_attention_weights", dict(weights=0, k=0, stride=0, max_k=0, total_k=0)),
])
def test_weights_of_no_keys_pass_the_checks(lib, name, kw):
    args = dict(abi.CALLS[name], **kw)
    entry, words = _lib.CALLS[name]
    for rc in (getattr(lib, name)(*args.values()), lib.mea_call(entry, words.pack(*args.values()))):
        assert rc in (_lib.MEA_ERR_CUDA, _lib.MEA_ERR_DEVICE)  # past the checks: there is no GPU
