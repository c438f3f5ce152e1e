"""What the binding of the epilogue and expert calls hands to the library (no GPU: tensors of the meta
device, which have shapes alone, and a library that records its calls)."""
import pytest
import torch

import bit_weight_quantized_tgemm_b200 as tg
from bit_weight_quantized_tgemm_b200 import binding

BIG = 2 ** 32 + 5  # 5, to a C int


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name == "tgemm_strerror":
            raise AttributeError(name)

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    lib = Recorder()
    monkeypatch.setattr(binding, "_lib", lib)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(binding, "_first", lambda t, dtype, name: 0)
    monkeypatch.setattr(binding, "_arg", lambda t, dtype, name, index: t.data_ptr())
    return lib.calls


def empty(*shape, dtype):
    return torch.empty(*shape, dtype=dtype, device="meta")


def weights(*lead, K=128):
    return empty(*lead, K // 4, dtype=torch.uint8), empty(*lead, K // 128, dtype=torch.float16)


@pytest.mark.parametrize("call", [
    lambda: tg.gemm_q2_ep(empty(BIG, 128, dtype=torch.bfloat16), *weights(8)),
    lambda: tg.gemm_q2_ep(empty(4, 128, dtype=torch.bfloat16), *weights(BIG)),
    lambda: tg.gemm_q2_grouped(empty(4, 128, dtype=torch.bfloat16), *weights(3, 1), empty(4, dtype=torch.int32),
                               rows=empty(BIG, dtype=torch.int32)),
    lambda: tg.gemm_q2_grouped(empty(BIG, 128, dtype=torch.bfloat16), *weights(3, 1), empty(4, dtype=torch.int32),
                               rows=empty(9, dtype=torch.int32)),
    lambda: tg.expert_sort(empty(BIG, 1, dtype=torch.int32), 8),
    lambda: tg.expert_combine(empty(9, 8, dtype=torch.bfloat16), empty(BIG, 1, dtype=torch.int32), empty(BIG, 1, dtype=torch.float32)),
    lambda: tg.expert_combine(empty(BIG, 8, dtype=torch.bfloat16), empty(9, 1, dtype=torch.int32), empty(9, 1, dtype=torch.float32)),
], ids=["x", "wq", "rows", "x of rows", "ids", "pos", "h"])
def test_sizes_past_a_c_int_are_refused(calls, call):
    with pytest.raises(tg.TgemmError) as e:
        call()
    assert e.value.status == tg.ETOOLARGE and not calls


def test_sizes_go_through_as_they_are(calls):
    tg.gemm_q2_ep(empty(7, 256, dtype=torch.bfloat16), *weights(8, K=256))
    tg.expert_sort(empty(7, 2, dtype=torch.int32), 8)
    assert [c[0] for c in calls] == ["tgemm_ep_workspace_size", "tgemm_q2_ep", "tgemm_expert_sort_workspace_size", "tgemm_expert_sort"]
    assert calls[1][1][5:8] == (7, 8, 256) and calls[3][1][1:4] == (7, 2, 8)
