"""The epilogue and expert kernels' sources (no GPU)."""
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parent.parent / "bit_weight_quantized_tgemm_b200" / "csrc"


@pytest.mark.parametrize("name", ["epilogue.cuh", "expert.cuh", "ep_small.cuh", "ep_tc.cuh"])
def test_read_only_loads_are_of_packed_weights_alone(name):
    """These kernels may be resident while the one before them writes their activations, plans and
    epilogue operands, and the read-only path (__ldg, ld.global.nc, const __restrict__) is for memory
    that nobody writes meanwhile.  Packed weights and scales go through ld_stream_v2 and ld_scale."""
    text = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    for helper in ("ld_stream_v2", "ld_scale"):
        text = re.sub(helper + r"\(const \w+\* p\) \{.*?\}\n", "", text, flags=re.S)
    assert not re.findall(r"__ldg|ld\.global\.nc|__restrict__", text)
    for arg in re.findall(r"\bld_scale\((.*?)\)", text) + re.findall(r"\bld_stream_v2\((.*?)\)", text):
        assert re.fullmatch(r"(src|q)( \+ \d+)?", arg), arg
