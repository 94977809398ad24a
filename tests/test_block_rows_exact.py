"""Block rows to both sides of what chooses their kernels."""
import pytest

torch = pytest.importorskip("torch")

from test_block_operators import check_block_codes  # noqa: E402
from test_operators import TYPES, act64, normal, padded  # noqa: E402

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("more", [-1, 0, 1])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dtype", ["BF16", "F16", "F32"])
@pytest.mark.parametrize("each", [8, 32])
def test_gated_act_blocks_to_both_sides_of_a_full_gpu(stmat, more, off, dtype, each):
    """So many blocks of 256 accesses an SM, one row fewer and one more, on and
    off the accesses' boundaries."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    m, c = each * sms + more, 256 * (4 if dtype == "F32" else 8) - off
    gate, up = (padded(normal(i, m, c, dtype=TYPES[dtype]), 2 * off, off) for i in (1, 2))
    y, scales = stmat.gated_act(gate, up, act="relu", dst="F8_E4M3", block=128)
    check_block_codes(y, scales, act64(gate.double(), "relu") * up.double())
