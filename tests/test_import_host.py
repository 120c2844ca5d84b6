"""The package on a torch without CUDA: it imports, its host objects work and a call says that its
tensors are not on a GPU."""
import os
import subprocess
import sys

CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)  # (a torch built without CUDA has none of them)
import memory_efficient_attention_b200 as mea
assert mea.alibi_slopes(8).shape == (8,)
assert mea.tree_mask([[-1, 0]]).tolist() == [[1], [3]]
kc, table = torch.zeros((2, 16, 1, 8)).half(), torch.zeros((1, 1), dtype=torch.int32)
cu = torch.tensor([0, 3], dtype=torch.int32)
for call in (lambda: mea.block_key_bounds(kc, table, cu, 3),
             lambda: mea.decode_paged(torch.zeros((1, 1, 8)).half(), kc, kc, table, cu, 3)):
    try:
        call()
    except mea.MeaError as e:
        assert e.rc == mea._lib.MEA_ERR_DEVICE
    else:
        raise AssertionError("no MeaError")
print("imported")
"""


def test_import_without_cuda_in_torch():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", CODE], cwd=root, capture_output=True, text=True,
                         timeout=300, env={**os.environ, "CUDA_VISIBLE_DEVICES": ""})
    assert res.returncode == 0 and "imported" in res.stdout, res.stderr[-2000:]
