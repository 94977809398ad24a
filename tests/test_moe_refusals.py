"""Operands that a mixture-of-experts layer could not use are refused, not
passed over."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

from test_block_edges import experts, machine, on  # noqa: E402, F401
from test_moe import moe_args  # noqa: E402


def test_scales_without_the_matrix_they_belong_to(stmat):
    a = moe_args(stmat, up__w=None)
    assert a.up.scale
    assert stmat.STATUS[stmat.lib().st_moe(C.byref(a), None)] == "ST_E_INVAL"
    assert "up" in stmat.lib().st_last_error().decode()
    need = C.c_uint64()
    assert stmat.STATUS[stmat.lib().st_moe_workspace(C.byref(a), C.byref(need))] == "ST_E_INVAL"
    a.up.scale = None
    assert stmat.STATUS[stmat.lib().st_moe_workspace(C.byref(a), C.byref(need))] == "ST_OK"


def test_binding_refuses_up_scale_without_up(stmat, machine):  # noqa: F811
    x = on(1, 4, 256)
    args = dict(experts(), up=None)
    with pytest.raises(stmat.StmatError) as e:
        stmat.moe(x, **args)
    assert e.value.status == "ST_E_INVAL" and "up_scale" in str(e.value) and machine.calls == []
    stmat.moe(x, **dict(args, up_scale=None))
    assert len(machine.calls) == 1
