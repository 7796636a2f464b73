"""Host-side checks of the training block's operators (no GPU needed): struct
mirrors, scratch sizes, and refusals before anything touches the device."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

from moe_routing_capacity_gb300 import abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_pooled_wave.h")


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(abi.LIB_PATH):
        from moe_routing_capacity_gb300 import build
        build.build()
    return abi.lib()


@pytest.mark.parametrize("struct,cls", [("moe_norm_t", abi.Norm),
                                        ("moe_rotary_table_t", abi.RotaryTable),
                                        ("moe_rotary_t", abi.Rotary),
                                        ("moe_attention_t", abi.Attention),
                                        ("moe_grad_tensor_t", abi.GradTensor)])
def test_struct_mirrors_match_header(struct, cls, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    fields = [f for f, _ in cls._fields_]
    src = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{HEADER}"', "int main(void) {",
           f'  printf("%zu\\n", sizeof({struct}));']
    src += [f'  printf("%zu\\n", offsetof({struct}, {f}));' for f in fields] + ["}"]
    (tmp_path / "s.c").write_text("\n".join(src))
    subprocess.run([cc, str(tmp_path / "s.c"), "-o", str(tmp_path / "s")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]


P = ctypes.c_void_p(0x10000)          # a 16-byte aligned address nobody reads
ODD = ctypes.c_void_p(0x10008)


def norm(**kw):
    c = abi.Norm(4, 64, 0, 0, 1.0, 1.0, 1e-6)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(d=0), dict(d=4), dict(d=63), dict(d=8200),
                                dict(res_f32=2), dict(gate_per_token=3), dict(alpha=math.inf),
                                dict(beta=math.nan), dict(eps=-1.0), dict(eps=math.nan)])
def test_norm_refuses_sizes(kw):
    L = abi.lib()
    assert L.moe_norm_residual(norm(**kw), P, P, None, P, P, P, P, None, None, None) == abi.MOE_EINVAL
    assert L.moe_norm_residual_backward(norm(**kw), P, P, P, P, None, P, P, P, P, P, P, None, P, P,
                                        P, 1 << 40, None) == abi.MOE_EINVAL


@pytest.mark.parametrize("i,v", [(1, None), (1, ODD), (0, None), (3, None), (4, None), (6, None),
                                 (0, ODD), (2, ODD), (5, ODD), (6, ODD)])
def test_norm_refuses_pointers(i, v):
    # b, r, gate, w_post, w_pre, y, n, rstd_post, rstd_pre
    a = [P, P, P, P, P, P, P, None, None]
    a[i] = v
    assert abi.lib().moe_norm_residual(norm(), *a, None) == abi.MOE_EINVAL


def test_norm_refuses_nothing_to_do_and_short_scratch():
    L = abi.lib()
    assert L.moe_norm_residual(norm(), None, P, None, None, None, P, None, None, None, None) == abi.MOE_EINVAL
    assert L.moe_norm_residual(norm(), P, P, None, P, None, None, None, None, None, None) == abi.MOE_EINVAL
    need = abi.norm_residual_workspace(4, 64)
    assert need == 4 * 2 * 64 * 4
    args = [P, P, P, P, None, P, P, P, P, P, P, None, P, P, P]
    assert L.moe_norm_residual_backward(norm(), *args, need - 1, None) == abi.MOE_ENOSPC
    for i in (2, 5, 7, 9, 10, 12, 13, 14):      # a tensor that belongs to the call is missing
        b = list(args)
        b[i] = None
        assert L.moe_norm_residual_backward(norm(), *b, need, None) == abi.MOE_EINVAL, i
    assert L.moe_norm_residual(norm(T=0), *[None] * 9, None) == abi.MOE_OK


def rotary(**kw):
    c = abi.Rotary(4, 2, 1, 64, 32, 0, 0, 100, 192, 64, 192, 64, 128, 64, 64, 64)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(hq=0), dict(hk=-1), dict(D=60), dict(D=8),
                                dict(D=2048), dict(rot_dim=8), dict(rot_dim=72), dict(rot_dim=40),
                                dict(interleaved=2), dict(inverse=-1), dict(table_rows=0),
                                dict(q_t=100), dict(q_h=32), dict(qo_t=64), dict(k_t=0),
                                dict(ko_t=4)])
def test_rotary_refuses_sizes(kw):
    assert abi.lib().moe_rotary(rotary(**kw), P, P, P, None, P, P, P, None) == abi.MOE_EINVAL


def test_rotary_refuses_pointers():
    L = abi.lib()
    q2, k2 = ctypes.c_void_p(0x20000), ctypes.c_void_p(0x30000)
    good = [P, P, P, None, q2, k2, P]
    for i, v in ((0, None), (0, ODD), (1, None), (2, None), (4, ODD), (5, None), (6, None)):
        a = list(good)
        a[i] = v
        assert L.moe_rotary(rotary(), *a, None) == abi.MOE_EINVAL, i
    # in place with other strides
    assert L.moe_rotary(rotary(), P, q2, P, None, P, k2, P, None) == abi.MOE_EINVAL
    assert L.moe_rotary(rotary(T=0), *[None] * 7, None) == abi.MOE_OK


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(rot_dim=1), dict(rot_dim=3), dict(scaling=4),
                                dict(base=1.0), dict(factor=0.5), dict(factor=2.0),
                                dict(magnitude=0.0), dict(scaling=2, rot_dim=2, factor=2.0),
                                dict(scaling=3, factor=2.0),
                                dict(scaling=3, factor=2.0, orig_len=10.0, beta_fast=1.0)])
def test_rotary_table_refuses(kw):
    c = abi.RotaryTable(8, 32, 0, 1e4, 1.0, 0.0, 32.0, 1.0, 1.0)
    for k, v in kw.items():
        setattr(c, k, v)
    assert abi.lib().moe_rotary_make_table(ctypes.byref(c), P, None) == abi.MOE_EINVAL


def attention(**kw):
    c = abi.Attention()
    c.T, c.n_seqs, c.n_heads, c.n_kv_heads, c.head_dim, c.scale = 10, 1, 4, 2, 64, 0.125
    for n, h in (("q", 4), ("k", 2), ("v", 2), ("o", 4), ("do", 4), ("dq", 4), ("dk", 2), ("dv", 2)):
        setattr(c, n + "_t", h * 64)
        setattr(c, n + "_h", 64)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(n_seqs=-1), dict(n_heads=0), dict(n_heads=5),
                                dict(n_kv_heads=0), dict(head_dim=0), dict(head_dim=12),
                                dict(head_dim=136), dict(scale=0.0), dict(scale=-1.0),
                                dict(scale=math.nan), dict(scale=math.inf), dict(reserved=1),
                                dict(T=1 << 31)])
def test_attention_refuses_sizes(kw):
    L = abi.lib()
    a, b = ctypes.c_int64(), ctypes.c_int64()
    c = attention(**kw)
    assert L.moe_attention_workspace(c, ctypes.byref(a), ctypes.byref(b)) == abi.MOE_EINVAL
    assert L.moe_attention_plan(c, P, P, 1 << 40, P, None) == abi.MOE_EINVAL
    assert L.moe_attention_forward(c, P, P, P, P, P, None, P, P, None) == abi.MOE_EINVAL
    assert L.moe_attention_backward(c, *[P] * 12, 1 << 40, P, None) == abi.MOE_EINVAL


@pytest.mark.parametrize("kw", [dict(q_t=255), dict(q_t=128), dict(k_h=32), dict(v_t=0),
                                dict(o_h=60), dict(k_t=-128), dict(q_t=1 << 40)])
def test_attention_refuses_strides(kw):
    L = abi.lib()
    assert L.moe_attention_forward(attention(**kw), P, P, P, P, P, None, P, P, None) == abi.MOE_EINVAL


def test_attention_refuses_pointers_and_short_scratch():
    L = abi.lib()
    a, b = ctypes.c_int64(), ctypes.c_int64()
    c = attention()
    assert L.moe_attention_workspace(c, ctypes.byref(a), ctypes.byref(b)) == abi.MOE_OK
    assert L.moe_attention_plan(c, P, P, a.value - 1, P, None) == abi.MOE_ENOSPC
    for args in ([None, P, 1 << 30, P], [P, ODD, 1 << 30, P], [P, P, 1 << 30, None]):
        assert L.moe_attention_plan(c, *args, None) == abi.MOE_EINVAL
    good = [P, P, P, P, P, None, P, P]
    for i, v in ((0, None), (1, ODD), (2, None), (3, None), (4, None), (5, ODD), (6, None), (7, None)):
        x = list(good)
        x[i] = v
        assert L.moe_attention_forward(c, *x, None) == abi.MOE_EINVAL, i
    for i in range(12):
        x = [P] * 12
        x[i] = None
        assert L.moe_attention_backward(c, *x, 1 << 40, P, None) == abi.MOE_EINVAL, i
    assert L.moe_attention_backward(c, *[P] * 12, b.value - 1, P, None) == abi.MOE_ENOSPC
    assert L.moe_attention_backward(attention(dk_t=100), *[P] * 12, 1 << 40, P, None) == abi.MOE_EINVAL
    assert L.moe_attention_forward(attention(T=0), *[None] * 8, None) == abi.MOE_OK


def test_grad_clip_refuses():
    L = abi.lib()
    need = ctypes.c_int64()
    assert L.moe_grad_clip_workspace(1, ctypes.byref(need)) == abi.MOE_OK

    def call(n=1, max_norm=1.0, norm=P, ws=P, ws_bytes=None, **kw):
        r = (abi.GradTensor * 1)()
        setattr(r[0], "in", 0x10000)
        r[0].out, r[0].numel = 0x20000, 5
        for k, v in kw.items():
            setattr(r[0], k, v)
        return L.moe_grad_clip(r, n, max_norm, norm, ws, need.value if ws_bytes is None else ws_bytes, None)

    for kw in (dict(n=-1), dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=math.nan),
               dict(norm=None), dict(ws=None), dict(ws=ODD), dict(numel=-1), dict(is_bf16=2),
               dict(out=None), dict(out=0x20002), dict(out=0x20001, is_bf16=1), dict(reserved=1),
               dict(n=(1 << 20) + 1)):
        assert call(**kw) == abi.MOE_EINVAL, kw
    assert call(ws_bytes=need.value - 1) == abi.MOE_ENOSPC
    assert L.moe_grad_clip(None, 0, 1.0, None, None, 0, None) == abi.MOE_OK


def test_python_checks_types_and_shapes():
    """Raised from the tensors alone, before the library is called."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    with pytest.raises(TypeError):
        abi.norm_residual(z(2, 8, dt=torch.float16), z(2, 8), None, z(8), z(8), z(2, 8), z(2, 8))
    with pytest.raises(ValueError):
        abi.norm_residual(z(3, 8), z(2, 8), None, z(8), z(8), z(2, 8), z(2, 8))
    with pytest.raises(ValueError):
        abi.norm_residual(None, z(2, 8), None, None, z(8), None, z(2, 8))    # not on the GPU
    with pytest.raises(TypeError):
        abi.rotary(z(2, 1, 16, dt=torch.float32), None, z(4, 8, 2), None, z(2, 1, 16), None, None)
    with pytest.raises(ValueError):
        abi.rotary_table(z(4, 8, 2, dt=torch.float32), scaling="sideways")
    with pytest.raises(TypeError):
        abi.GradSet([z(4, dt=torch.float64)])
    with pytest.raises(ValueError):
        abi.GradSet([z(4)], [])
