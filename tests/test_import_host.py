"""The package without a CUDA torch (no GPU)."""
import subprocess
import sys
from pathlib import Path


def test_imports_with_a_torch_that_has_no_cuda():
    """Such a torch lacks the CUDA entries of torch._C: the import works, the calls refuse CPU tensors."""
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import bit_weight_quantized_tgemm_b200 as tg
x = torch.zeros(4, 256, dtype=torch.bfloat16)
wq, d = torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.float16)
ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
for call in (lambda: tg.gemm_q2_ep(x, wq, d), lambda: tg.gemm_q2_grouped(x, wq[None], d[None], ids[0]),
             lambda: tg.expert_sort(ids, 8), lambda: tg.expert_combine(x, ids, w)):
    try:
        call()
    except ValueError as e:
        assert "CUDA tensor" in str(e)
    else:
        raise AssertionError("not refused")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parent.parent, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
