"""GPU: rows of a norm with a NaN, to 8 bits: all of the row reads back as NaN, blocks of zeros too."""
import math

import pytest

import layer_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("block", [0, 32, 64, 128])
@pytest.mark.parametrize("x,res", [("f32", None), ("bf16", "f32")])
@pytest.mark.parametrize("width", [1, 47, 64, 131, 256, 1000, 5003, 20000, 40003])
def test_nan_row(x, res, width, block):
    """Rows of one NaN and otherwise zeros, of zeros under a NaN in the residual, of a gain that is zero; beside rows of zeros and
    of numbers, which stay as they are."""
    from kv_cached_qwen3_gb300.norm import rms_norm
    rows = ref.rnd(1, 5, width)
    rows[0] = rows[1] = rows[2] = 0
    rows[0, 0] = math.nan
    rows[1, width - 1] = math.nan
    rows[4, width // 2] = math.nan
    xs = rows.to(DT[x]).cuda()
    r = None if res is None else torch.zeros(5, width, dtype=DT[res], device="cuda")
    for gain in (torch.ones(width), torch.zeros(width)):
        y, s, scales = rms_norm(xs, gain.cuda(), residual=r, out_dtype=torch.float8_e4m3fn, block=block)
        v = y.float().cpu() * ref.by_block(scales.cpu(), block, width)
        for row in (0, 1, 4):
            assert v[row].isnan().all(), (row, v[row])
        assert (v[2] == 0).all() and v[3].isfinite().all()
    if r is not None:
        assert s[2].abs().max() == 0
        y, _, scales = rms_norm(torch.zeros_like(xs), torch.ones(width).cuda(), residual=rows.to(DT[res]).cuda(), out_dtype=torch.float8_e4m3fn,
                                block=block)
        assert (y.float().cpu() * ref.by_block(scales.cpu(), block, width))[[0, 1, 4]].isnan().all()


@pytest.mark.parametrize("width", [64, 131])
def test_rows_of_zeros_without_eps(width):
    """max|s gain| of 0 stores zeros whatever the norm's factor, infinity too."""
    from kv_cached_qwen3_gb300.norm import rms_norm
    y, _, scales = rms_norm(torch.zeros(3, width).cuda(), torch.ones(width).cuda(), eps=0.0, out_dtype=torch.float8_e4m3fn, block=32)
    assert (y.float() == 0).all() and (scales == 0).all()
