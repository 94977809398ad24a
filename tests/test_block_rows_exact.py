"""Block rows digit for digit, and to both sides of what chooses their kernels."""
import pytest

torch = pytest.importorskip("torch")

from test_block_operators import blocks_of, check_block_codes  # noqa: E402
from test_operators import TYPES, act64, normal, padded  # noqa: E402

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("m,c", [(3, 128), (64, 4096), (40, 1111), (5, 20480)])
@pytest.mark.parametrize("dtype", ["BF16", "F32"])
def test_scales_and_codes_are_the_formulas(stmat, m, c, dtype):
    """Values as they are: a scale is the correctly rounded quotient of the
    block's largest by 448 (2^-126 at least), a code the rounded product of the
    value and the correctly rounded inverse.  (Quotients and products of
    binary32 numbers in binary64, rounded once more, are rounded correctly.)"""
    g = torch.Generator().manual_seed(c)
    power = torch.randint(-120, 120, (m, blocks_of(c)), generator=g).float()
    power[0, 0] = -140
    x = normal(m, m, c) * torch.exp2(power).repeat_interleave(128, 1)[:, :c].cuda()
    x = x.to(TYPES[dtype])
    y, scales = stmat.gated_act(x, act="none", dst="F8_E4M3", block=128)
    v = torch.nn.functional.pad(x.double(), (0, blocks_of(c) * 128 - c)).reshape(m, -1, 128)
    want = (v.abs().amax(2) / 448).float().clamp_min(2.0 ** -126)
    assert torch.equal(scales, want)
    inverse = (1.0 / want.double()).float().double()
    codes = (v * inverse[..., None]).float().clamp(-448, 448).to(torch.float8_e4m3fn).reshape(m, -1)[:, :c]
    assert torch.equal(y.float(), codes.float())


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
