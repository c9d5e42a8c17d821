"""Sizes at the end of what the gated delta rule's kernels count in 32 bits, without a GPU."""
import ctypes

import pytest

pytest.importorskip("torch")


@pytest.mark.parametrize("T", [(1 << 31) - 1, (1 << 31) - 1023])
@pytest.mark.parametrize("packed", [False, True])
def test_longest_sequence(T, packed):
    import rwkv_linear_attention_wkv_b200 as W
    from rwkv_linear_attention_wkv_b200.gdr import GdrProblem
    ok = 4096
    p = GdrProblem(1, T, 1, 1, 64, 1, ok if packed else None, 1, 1.0, None, 0)
    assert W.lib.wkv_gdr_forward(ctypes.byref(p), *[ok] * 6, None, None, None) == 5
    assert W.lib.wkv_gdr_forward_workspace_bytes(ctypes.byref(p)) == 0
    assert W.lib.wkv_gdr_checkpoint_bytes(ctypes.byref(p)) == 0
