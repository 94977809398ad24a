"""Edges of the calls of block_linear, moe and the rows with block scales: the
GPU they run on (stand-ins for tensors of several GPUs, on the CPU), offsets
beyond 32 bits, sizes that no other test reaches, the example."""
import importlib.util
import math
import os
import types

import pytest

torch = pytest.importorskip("torch")

from test_block_operators import check_block_codes, blocks_of, operands, product64  # noqa: E402
from test_moe import check, layer  # noqa: E402
from test_operator_edges import Machine, Stream, Tensor  # noqa: E402
from test_operators import act64, check_linear, check_values, norm64, normal  # noqa: E402

gpu = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture
def machine(stmat, monkeypatch):
    m = Machine(stmat)
    m.torch = types.SimpleNamespace(**vars(m.torch), int32=torch.int32)
    for op in ("rms_norm_blocks", "gated_act_blocks", "block_linear", "moe"):
        setattr(m, op, lambda args, stream, op=op: m.calls.append((op, m.current, stream)) or 0)
    m.moe_workspace = lambda args, to: 0
    m.moe_spaces = {}
    monkeypatch.setattr(stmat, "_OPS", m)
    return m


def on(device, *shape, dtype=torch.bfloat16):
    return Tensor(shape, dtype, device)


def f32(device, *shape):
    return on(device, *shape, dtype=torch.float32)


def experts(device=1, scale=1):
    """The operands of a layer of 4 experts of 256 -> 128."""
    return dict(router=on(device, 4, 256), gate=on(device, 4, 128, 256, dtype=E4M3), up=on(device, 4, 128, 256, dtype=E4M3),
                down=on(device, 4, 256, 128, dtype=E4M3), gate_scale=f32(scale, 4, 1, 2), up_scale=f32(scale, 4, 1, 2),
                down_scale=f32(scale, 4, 2, 1), top_k=2)


def test_a_call_runs_on_its_operands_gpu(stmat, machine):
    x, x8, w8 = on(1, 4, 256), on(1, 4, 256, dtype=E4M3), on(1, 8, 256, dtype=E4M3)
    for current in (0, 1):
        machine.current = current
        for name, call in (("rms_norm_blocks", lambda **k: stmat.rms_norm(x, dst="F8_E4M3", block=128, **k)),
                           ("gated_act_blocks", lambda **k: stmat.gated_act(x, x, dst="F8_E4M3", block=128, **k)),
                           ("block_linear", lambda **k: stmat.block_linear(x8, w8, f32(1, 4, 2), f32(1, 1, 2), **k)),
                           ("moe", lambda **k: stmat.moe(x, **experts(), **k))):
            for kw in ({}, {"stream": 101}, {"stream": Stream(101, 1)}):
                machine.calls.clear()
                got = call(**kw)
                assert machine.calls == [(name, 1, 101)] and machine.current == current
                assert all(t is None or t.device == 1 for t in (got if isinstance(got, tuple) else (got,)))


def test_operands_and_streams_of_several_gpus_are_refused(stmat, machine):
    x, x8, w8, xs, ws = on(1, 4, 256), on(1, 4, 256, dtype=E4M3), on(1, 8, 256, dtype=E4M3), f32(1, 4, 2), f32(1, 1, 2)
    for far in (0, -1):
        calls = [lambda **k: stmat.block_linear(x8, on(far, 8, 256, dtype=E4M3), xs, ws, **k),
                 lambda **k: stmat.block_linear(x8, w8, f32(far, 4, 2), ws, **k), lambda **k: stmat.block_linear(x8, w8, xs, f32(far, 1, 2), **k),
                 lambda **k: stmat.block_linear(x8, w8, xs, ws, bias=on(far, 8), **k),
                 lambda **k: stmat.block_linear(x8, w8, xs, ws, residual=on(far, 4, 8), **k),
                 lambda **k: stmat.block_linear(x8, w8, xs, ws, out=on(far, 4, 8), **k),
                 lambda **k: stmat.rms_norm(x, on(far, 256), dst="F8_E4M3", block=128, **k),
                 lambda **k: stmat.gated_act(x, on(far, 4, 256), dst="F8_E4M3", block=128, **k),
                 lambda **k: stmat.moe(x, **experts(scale=far), **k), lambda **k: stmat.moe(x, **experts(), out=on(far, 4, 256), **k),
                 lambda **k: stmat.moe(x, **experts(), residual=on(far, 4, 256), **k),
                 lambda **k: stmat.moe(x, **experts(), router_bias=f32(far, 4), **k)]
        for name in ("router", "gate", "up", "down"):
            other = dict(experts(), **{name: experts(far)[name]})
            calls.append(lambda other=other, **k: stmat.moe(x, **other, **k))
        for current in (0, 1):
            machine.current = current
            for i, call in enumerate(calls):
                for kw in ({}, {"stream": Stream(101, 1)}):
                    with pytest.raises(stmat.StmatError) as e:
                        call(**kw)
                    assert e.value.status == "ST_E_INVAL" and "GPU" in str(e.value), i
    for call in (lambda s: stmat.block_linear(x8, w8, xs, ws, stream=s), lambda s: stmat.moe(x, **experts(), stream=s)):
        with pytest.raises(stmat.StmatError) as e:
            call(Stream(100, 0))
        assert e.value.status == "ST_E_INVAL" and "GPU" in str(e.value)
    assert machine.calls == []


# ------------------------------------------------------ far offsets, on a GPU

def far_buffer(nbytes):
    if torch.cuda.mem_get_info()[0] < 2 * nbytes:
        pytest.skip("needs more device memory")
    return torch.zeros(nbytes, dtype=torch.uint8, device="cuda")


@gpu
@pytest.mark.parametrize("m", [3, 200])
def test_block_linear_offsets_beyond_32_bits(stmat, m):
    """Weight rows and rows of y that start more than 2^32 elements in."""
    n, k, ld = 130, 200, 1 << 26
    buf = far_buffer(n * ld)
    x, w, xs, ws = operands(m, n, k)
    far = buf.view(E4M3).as_strided((n, k), (ld, 1))
    far.copy_(w)
    want, slack = product64(x, w, xs, ws)
    check_linear(stmat.block_linear(x, far, xs, ws, dst="F32"), want, slack)
    del far, w
    x, w, xs, ws = operands(n, 40, k)
    out = buf.view(torch.bfloat16).as_strided((n, 40), (ld // 2, 1), 1024)
    stmat.block_linear(x, w, xs, ws, out=out)
    want, slack = product64(x, w, xs, ws)
    check_linear(out, want, slack)


@gpu
def test_block_rows_offsets_beyond_32_bits(stmat):
    m, c, ld = 5, 1000, (1 << 30) + 8
    buf = far_buffer(2 * (m * ld + 4096))
    src, w = normal(1, m, c, dtype=torch.bfloat16), normal(2, c)
    for extra in (0, 1):    # rows on 16-byte boundaries, and off them
        x = buf.view(torch.bfloat16).as_strided((m, c), (ld + extra, 1), extra)
        x.copy_(src)
        y, scales, _ = stmat.rms_norm(x, w, dst="F8_E4M3", block=128)
        check_block_codes(y, scales, norm64(src, None, w, 1e-5)[1])
        y, scales = stmat.gated_act(x, x, dst="F8_E4M3", block=128)
        check_block_codes(y, scales, act64(src.double(), "silu") * src.double(), slack=80 * 2.0 ** -23)


@gpu
def test_moe_offsets_beyond_32_bits(stmat):
    """Experts more than 2^31 elements apart."""
    t, e, k, h, i, step = 9, 4, 3, 256, 200, (1 << 31) + 4096
    args, weights = layer(3, t, e, h, i)
    buf = far_buffer(e * step).view(E4M3)
    for j, name in enumerate(("gate", "up", "down")):
        w = args[name]
        far = buf.as_strided(w.shape, (step, w.stride(1), 1), j << 20)
        far.copy_(w)
        args[name] = far
    check(stmat, args, weights, k)


# ------------------------------------------------------------- other sizes

@gpu
@pytest.mark.parametrize("m,n,k", [(64, 4096, 256), (65, 130, 8200), (8, 14336, 128), (256, 128, 16000), (4000, 70, 300), (130, 20000, 128)])
def test_block_linear_sizes_of_every_choice(stmat, m, n, k):
    x, w, xs, ws = operands(m, n, k)
    r = normal(5, m, n, dtype=torch.bfloat16)
    want, slack = product64(x, w, xs, ws, act="silu", r=r)
    check_linear(stmat.block_linear(x, w, xs, ws, act="silu", residual=r), want, slack + 2.0 ** -20 * want.abs())


@gpu
@pytest.mark.parametrize("m,n", [(300, 520), (257, 600), (1000, 4104), (2560, 1032)])
@pytest.mark.parametrize("dst", ["BF16", "F16"])
def test_block_linear_residuals_of_whole_and_partial_tiles(stmat, m, n, dst):
    """Tiles written and residuals read by TMA: rows of y and the residual at
    strides of their own, in place, and nothing written outside y."""
    x, w, xs, ws = operands(m, n, 384)
    dt = torch.bfloat16 if dst == "BF16" else torch.float16
    buf = torch.full((m + 2, n + 16), 77.0, device="cuda").to(dt)
    y, r = buf[1:-1, 8:-8], normal(5, m, n + 24, dtype=dt)[:, :n]
    for width in (192, 256):
        want, slack = product64(x, w, xs, ws, r=r)
        stmat.block_linear(x, w, xs, ws, residual=r, out=y, form=("dense", width, 1))
        check_linear(y, want, slack)
        first = y.clone()
        y.copy_(r)
        stmat.block_linear(x, w, xs, ws, residual=y, out=y, form=("dense", width, 1))
        assert torch.equal(y, first)
        edge = torch.ones_like(buf, dtype=torch.bool)
        edge[1:-1, 8:-8] = False
        assert (buf[edge].float() == 77).all()


@gpu
@pytest.mark.parametrize("t", [1, 8, 33, 64])
@pytest.mark.parametrize("x_kind,w_kind", [("F16", "F8_E5M2"), ("F16", "F8_E4M3"), ("BF16", "BF16")])
def test_moe_with_one_expert_and_all_of_them(stmat, t, x_kind, w_kind):
    """No choice at all: one expert, and every expert of every token; runs of
    hidden and inter that end early."""
    args, weights = layer(t, t, 1, 136, 264, x_kind, w_kind)
    check(stmat, args, weights, 1)
    args, weights = layer(t, t, 7, 136, 264, x_kind, w_kind)
    check(stmat, args, weights, 7, normalize=False)


@gpu
def test_moe_values_between_the_products_far_from_one(stmat):
    """h of 2^-60 and 2^60: its runs' scales are its own (F16 experts too,
    whose range it leaves)."""
    for w_kind, x_kind in (("F8_E4M3", "BF16"), ("BF16", "BF16"), ("F16", "F16")):
        args, weights = layer(5, 4, 5, 256, 256, x_kind, w_kind)
        for power in (-60, 60):
            y, chosen, p = stmat.moe(**args, top_k=2, act="none", factor=2.0 ** power, dst="F32")
            one = stmat.moe(**args, top_k=2, act="none", dst="F32")[0]
            check_values(y, one.double() * 2.0 ** power, slack=2.0 ** -20, extra=2.0 ** (power - 18) * one.double().abs().amax())
            assert math.isfinite(float(y.abs().max()))


@gpu
def test_block_fp8_moe_example():
    """A checkpoint's experts through the loader and the layer.  The sum's
    rounding to BF16 is off by at most 2^-8 of it; h's columns by 2^-12 of a term,
    of which the 320 of a sum are about sqrt(320) = 2^4.2 times it: under 2^-6 in
    all."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "block_fp8_moe.py")
    spec = importlib.util.spec_from_file_location("block_fp8_moe", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    found = example.main(hidden=512, inter=320, experts=12, top_k=3, tokens=(1, 13, 64))
    assert set(found) == {1, 13, 64} and all(0 < v < 2.0 ** -6 for v in found.values()), found


@gpu
def test_no_wait_gave_up(stmat):
    torch.cuda.synchronize()
    assert stmat.static_check() == 0 and blocks_of(129) == 2
