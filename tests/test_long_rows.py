"""Norms of rows of 2^20 columns and more: what the sum of squares may be off by
does not grow with the row.

Tolerance: a thread's run of 64 squares is off by at most 64 2^-24 of it, the
runs' sum by 2^-24, the block's tree of 10 additions by 10 2^-24, the mean's
division and eps by 2 2^-24: 77 2^-24 of the mean, half of that of its root;
rsqrtf's two units of the last place 4 2^-24, the product with it and the quotient
by 448 2 2^-24: 45 2^-24 in all, and the second orders.  (Rows of equal values
are the worst: the roundings of one long chain all go the same way, 120 to 2000
2^-24 of the root at these sizes.)"""
import pytest

torch = pytest.importorskip("torch")

from test_block_operators import blocks_of, check_block_codes  # noqa: E402
from test_operators import TYPES, check_values, norm64, normal  # noqa: E402

gpu = pytest.mark.gpu
LONG = 46 * 2.0 ** -24
# Columns, and the value that fills the row (eight bits or fewer).
EQUAL = [(1 << 20, 1.3359375), (1 << 23, 1.7109375), ((1 << 23) + 5, 1.2265625), ((1 << 25) + 130, 0.703125)]


@gpu
@pytest.mark.parametrize("c,value", EQUAL)
@pytest.mark.parametrize("dtype", ["BF16", "F16", "F32"])
def test_norm_blocks_of_equal_values(stmat, c, value, dtype):
    x = torch.full((1, c), value, dtype=TYPES[dtype], device="cuda")
    for residual in (None, torch.zeros_like(x)):
        y, scales, h = stmat.rms_norm(x, residual=residual, eps=0.0, dst="F8_E4M3", block=128)
        want = 1.0 / 448    # every value is 1
        assert scales.shape == (1, blocks_of(c)) and ((scales.double() - want).abs() <= LONG * want).all()
        assert (y.float() == 448).all()
        assert h is None or torch.equal(h, x)


@gpu
@pytest.mark.parametrize("m,c", [(2, 65536), (3, 65537), (2, 70001), (1, (1 << 21) + 77)])
@pytest.mark.parametrize("dtype", ["BF16", "F32"])
def test_norm_blocks_of_long_rows(stmat, m, c, dtype):
    x, r, w = normal(m, m, c, dtype=TYPES[dtype]), normal(m + 1, m, c, dtype=TYPES[dtype]), normal(3, c, dtype=TYPES[dtype])
    for residual, weight in ((r, w), (None, None)):
        y, scales, _ = stmat.rms_norm(x, weight, residual=residual, dst="F8_E4M3", block=128)
        check_block_codes(y, scales, norm64(x, residual, weight, 1e-5)[1], slack=LONG)


@gpu
def test_norm_blocks_of_long_rows_that_leave_binary32(stmat):
    """A sum of squares that is infinite makes the row's factor 0 (and an
    infinity in it NaN), as in short rows; a NaN makes the row NaN."""
    for c in (20000, 100000, 1 << 20):
        x = torch.full((3, c), 1.0, device="cuda")
        x[0] = 1e19
        x[1, 9] = float("inf")
        x[2, c - 1] = float("nan")
        y, scales, _ = stmat.rms_norm(x, dst="F8_E4M3", block=128)
        assert (y[0].float() == 0).all() and (scales[0] == 2.0 ** -126).all()
        assert torch.isnan(y[1, 9].float()) and (y[1, 128:].float() == 0).all() and (scales[1, 1:] == 2.0 ** -126).all()
        assert torch.isnan(y[2].float()).all() and torch.isnan(scales[2]).all()


@gpu
@pytest.mark.parametrize("c,value", EQUAL)
@pytest.mark.parametrize("dtype", ["BF16", "F16", "F32"])
@pytest.mark.parametrize("offset", [0, 1])
def test_norm_of_equal_values(stmat, c, value, dtype, offset):
    """One scale a row, or none; rows on and off the accesses' boundaries."""
    x = torch.full((1, c + offset), value, dtype=TYPES[dtype], device="cuda")[:, offset:]
    y, _, _ = stmat.rms_norm(x, eps=0.0, dst="F32")
    assert ((y.double() - 1.0).abs() <= LONG).all()
    y, scales, h = stmat.rms_norm(x, residual=torch.zeros_like(x), eps=0.0, dst="F8_E4M3")
    assert scales.shape == (1,) and ((scales.double() * 448 - 1.0).abs() <= LONG).all()
    assert (y.float() == 448).all() and torch.equal(h, x)


@gpu
@pytest.mark.parametrize("m,c", [(2, 65536), (3, 65537), (2, 70001), (1, (1 << 21) + 77)])
@pytest.mark.parametrize("dtype", ["BF16", "F32"])
def test_norm_of_long_rows(stmat, m, c, dtype):
    x, r, w = normal(m, m, c, dtype=TYPES[dtype]), normal(m + 1, m, c, dtype=TYPES[dtype]), normal(3, c, dtype=TYPES[dtype])
    for residual, weight in ((r, w), (None, None)):
        y, _, _ = stmat.rms_norm(x, weight, residual=residual, dst="F32")
        check_values(y, norm64(x, residual, weight, 1e-5)[1], slack=LONG)


@gpu
def test_norm_of_long_rows_that_leave_binary32(stmat):
    for c in (20000, 100000, 1 << 20):
        x = torch.full((3, c), 1.0, device="cuda")
        x[0] = 1e19
        x[1, 9] = float("inf")
        x[2, c - 1] = float("nan")
        y, _, _ = stmat.rms_norm(x)
        assert (y[0] == 0).all() and torch.isnan(y[1, 9]) and (y[1, 10:] == 0).all() and torch.isnan(y[2]).all()
        y, scales = stmat.gated_act(x, act="none", dst="F8_E4M3")
        # (A tensor's division by a number is torch's product with its inverse; this one is rounded correctly.)
        assert scales[0] == (x[0, 0].double() / 448).float() and scales[1] == float("inf") and torch.isnan(scales[2])
