"""CPU: a rotation's plan lies where its kernels run."""
import pytest


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_no_plan_without_cuda(device):
    from kv_cached_qwen3_gb300 import build
    from kv_cached_qwen3_gb300.rotary import Rotary
    build.build()
    with pytest.raises(ValueError, match="CUDA"):
        Rotary(64, device=device)
