"""Argument checks of the 8-bit expert operators and the balance loss, on the
CPU: every call here is refused before anything touches CUDA."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_reference as R
import mixture_experts_layer_53_b200 as M
from mixture_experts_layer_53_b200 import build as B

A = ctypes.c_void_p(0x10000)    # never dereferenced
OFF = ctypes.c_void_p(0x10008)  # not on a 16-byte boundary
ODD = ctypes.c_void_p(0x10002)  # not on a 4-byte boundary
WS = ctypes.c_void_p(0x100000)
BIG = ctypes.c_size_t(1 << 50)
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.library()


@pytest.mark.parametrize("args,code", [
    ((2, A, 4, 64, A, A), 1), ((0, A, -1, 64, A, A), 1), ((0, A, 4, 0, A, A), 1), ((0, A, 4, 24, A, A), 2), ((0, A, 4, 2 ** 30 + 16, A, A), 2),
    ((0, A, 2 ** 31, 64, A, A), 2), ((1, None, 4, 64, A, A), 1), ((1, OFF, 4, 64, A, A), 1),
    ((1, A, 4, 64, None, A), 1), ((1, A, 4, 64, A, ODD), 1), ((1, None, 0, 64, None, None), 0),
])
def test_quantize_rows(lib, args, code):
    assert lib.moe_quantize_rows(*args, None) == code


@pytest.mark.parametrize("args,code", [
    ((2, A, 1, 64, 64, 0, A, A), 1), ((0, A, 0, 64, 64, 0, A, A), 1), ((0, A, 1, 64, 0, 0, A, A), 1),
    ((0, A, 1, 64, 64, 2, A, A), 1), ((0, A, 1, 72, 64, 0, A, A), 2), ((0, A, 1, 64, 72, 0, A, A), 2),
    ((0, OFF, 1, 64, 64, 0, A, A), 1), ((0, A, 1, 64, 64, 1, None, A), 1), ((0, A, 1, 64, 64, 1, A, None), 1),
    ((0, A, 2 ** 31 - 1, 256, 64, 0, A, A), 2),
])
def test_quantize_weights(lib, args, code):
    assert lib.moe_quantize_weights(*args, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), 1), (dict(n=0), 1), (dict(k=0), 1), (dict(E=0), 1), (dict(E=257), 2), (dict(n=40), 2),
    (dict(k=40), 2), (dict(rows=2 ** 31), 2), (dict(dt=2), 1), (dict(any=2), 1), (dict(a=None), 1), (dict(a=OFF), 1), (dict(asc=None), 1), (dict(asc=ODD), 1), (dict(wsc=ODD), 1),
    (dict(off=None), 1), (dict(off=ctypes.c_void_p(0x10002)), 1), (dict(n=2 ** 30 + 16), 2), (dict(k=2 ** 30 + 16), 2),
    (dict(w=OFF), 1), (dict(wsc=None), 1), (dict(out=None), 1), (dict(out=OFF), 1),
    (dict(rows=0, a=None, asc=None, out=None), 0),
])
def test_matmul(lib, change, code):
    a = dict(rows=4, n=64, k=64, E=2, a=A, asc=A, off=A, w=A, wsc=A, any=0, dt=1, out=A)
    a.update(change)
    assert lib.moe_expert_matmul_fp8(*a.values(), None, None) == code


def test_ffn(lib):
    cfg = lambda **kw: M.make_config(**{**dict(N=8, d_model=64, d_ff=96, E=4, k=2, act="swiglu", dtype="bf16"), **kw})
    w = lambda **kw: M.Fp8Experts(**{**{n: 0x10000 for n in ("W1", "W1_scales", "W3", "W3_scales", "W2", "W2_scales")}, **kw})
    size = lambda c: lib.moe_expert_ffn_fp8_workspace_size(ctypes.byref(c))
    call = lambda c, e, x=A, off=A, y=A, ws=WS, n=BIG: lib.moe_expert_ffn_fp8(
        ctypes.byref(c), x, off, ctypes.byref(e) if e is not None else None, y, None, ws, n, None)
    assert size(cfg()) > 16 * (64 + 96)
    for bad in (dict(dtype="f32"), dict(d_model=72), dict(d_ff=72)):
        assert size(cfg(**bad)) == 0 and call(cfg(**bad), w()) == 2
    assert size(cfg(k=5)) == 0 and call(cfg(k=5), w()) == 1
    for name in ("W1", "W1_scales", "W3", "W3_scales", "W2", "W2_scales"):
        bad = 0x10002 if name.endswith("scales") else 0x10008
        assert call(cfg(), w(**{name: None})) == 1 and call(cfg(), w(**{name: bad})) == 1
    assert call(cfg(), w(b1=0x10000)) == 1                    # a hidden bias with SwiGLU
    assert call(cfg(act="gelu"), w()) == 1                    # W3 with GELU
    assert call(cfg(), w(b2=0x10008)) == 1 and call(cfg(), w(any_scales=-1)) == 1
    assert call(cfg(), None) == 1 and call(cfg(), w(), x=None) == 1 and call(cfg(), w(), off=None) == 1
    assert call(cfg(), w(), y=OFF) == 1
    assert call(cfg(), w(), ws=None) == 4 and call(cfg(), w(), ws=OFF) == 4
    assert call(cfg(), w(), n=ctypes.c_size_t(size(cfg()) - 1)) == 4
    assert call(cfg(N=0), w(), x=None, y=None) == 0


@pytest.mark.parametrize("change,code", [
    (dict(dt=2), 1), (dict(scores=2), 1), (dict(z=None), 1), (dict(z=OFF), 1), (dict(ids=None), 1), (dict(N=-1), 1),
    (dict(E=0), 1), (dict(E=257), 2), (dict(k=0), 1), (dict(k=9), 1), (dict(E=64, k=17), 2), (dict(S=0), 1),
    (dict(seq=None, S=3), 1), (dict(loss=None), 1), (dict(counts=None), 1), (dict(weight=None), 1), (dict(ws=None), 4),
    (dict(loss=ctypes.c_void_p(0x10002)), 1), (dict(ids=ctypes.c_void_p(0x10001)), 1), (dict(seq=ctypes.c_void_p(0x10003)), 1),
    (dict(ws=OFF), 4), (dict(size=ctypes.c_size_t(8)), 4), (dict(N=2 ** 31 - 1, k=2), 2),
])
def test_balance_loss(lib, change, code):
    a = dict(dt=0, scores=0, z=A, ids=A, seq=A, mask=None, N=64, E=8, k=2, S=4, loss=A, counts=A, weight=A, status=None,
             ws=WS, size=BIG)
    a.update(change)
    assert lib.moe_balance_loss(*a.values(), None) == code


@pytest.mark.parametrize("change,code", [
    (dict(dt=3), 1), (dict(scores=-1), 1), (dict(z=None), 1), (dict(E=300), 2), (dict(seq=None), 1),
    (dict(counts=None), 1), (dict(weight=None), 1), (dict(coef=F(float("nan"))), 1), (dict(dz=None), 1),
    (dict(dz=OFF), 1), (dict(dloss=ctypes.c_void_p(0x10002)), 1), (dict(N=0, z=None, dz=None), 0),
])
def test_balance_loss_backward(lib, change, code):
    a = dict(dt=0, scores=0, z=A, seq=A, mask=None, N=64, E=8, S=4, counts=A, weight=A, coef=F(1.0), dloss=None, dz=A)
    a.update(change)
    assert lib.moe_balance_loss_backward(*a.values(), None) == code


def test_balance_workspace(lib):
    size = lib.moe_balance_loss_workspace_size
    assert size(0, 8, 1) > 0 and size(4096, 256, 1) < size(4096, 256, 512)
    assert size(-1, 8, 1) == 0 and size(64, 0, 1) == 0 and size(64, 257, 1) == 0 and size(64, 8, 0) == 0


def test_binding_refuses_host_and_wrong_tensors():
    with pytest.raises(ValueError, match="CUDA device"):
        M.moe_quantize_rows(torch.zeros(4, 64))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        M.moe_quantize_rows(torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="rows, cols"):
        M.moe_quantize_weights(torch.zeros(4, 64))
    with pytest.raises(ValueError, match="logits"):
        M.moe_balance_loss(torch.zeros(8), torch.zeros(8, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="S \\+ 1"):
        M.moe_balance_loss(torch.zeros(8, 4), torch.zeros(8, 1, dtype=torch.int32),
                           seq_offsets=torch.zeros(1, dtype=torch.int32))


def test_fp8_experts_layout_matches_header(tmp_path):
    import os
    import subprocess
    src = tmp_path / "probe.c"
    names = [f for f, _ in M.Fp8Experts._fields_]
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "moe.h"\nint main(void) { printf("%zu", sizeof(moe_fp8_experts));'
                   + "".join(f'printf(" %zu", offsetof(moe_fp8_experts, {n}));' for n in names) + "return 0; }\n")
    exe = tmp_path / "probe"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(B.ROOT, "include"), str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)], text=True).split()]
    assert got == [ctypes.sizeof(M.Fp8Experts)] + [getattr(M.Fp8Experts, n).offset for n in names]


def test_reference_rounding_is_e4m3():
    """The reference's grid against torch's conversion, at every bf16 value in range and around each border."""
    v = torch.arange(0, 0x4400, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    v = torch.cat([v, torch.nextafter(v, torch.tensor(1e9)), torch.nextafter(v, torch.tensor(-1e9))])
    v = v[v.abs() <= 448]
    want = v.to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.e4m3_round(v.double().numpy()), want)
    s = R.scale_of([0.0, 448.0, np.nextafter(448.0, 1e3), 1.0, 3.0e38])
    assert list(s[:4]) == [2.0 ** -126, 1.0, 2.0, 2.0 ** -8] and 3.0e38 <= 448 * s[4] < 2 * 3.0e38
