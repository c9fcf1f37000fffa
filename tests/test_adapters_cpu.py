"""Host-side checks of the adapter, gated-activation and input-gradient entries: what
they refuse before any launch, and their workspace sizes (no GPU needed)."""
import ctypes
import os
import re

import pytest

from w8_a8_quantized_b200 import aq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARG, SHAPE, WORKSPACE = -1, -2, -5


def lora(**kw):
    v = dict(N=128, K=256, L=2, R=24, max_rank=16, a=16, bt=16, off=16, scale=16)
    v.update(kw)
    return ctypes.byref(aq.AqLoraStruct(**v))


def apply(ad=None, x=16, ldx=256, ids=16, M=4, y=16, ldy=128, out=16, ldo=128, dtype=0, s=16, ws=16, n=1 << 30):
    return aq.lib().aq_lora_apply(ad or lora(), x, ldx, ids, M, y, ldy, out, ldo, dtype, s, ws, n, None)


def backward(ad=None, dy=16, ldd=128, ids=16, M=4, s=16, x=16, ldx=256, sx=16, da=16, dbt=16, add=16, ldadd=256, dx=16,
             lddx=256, dtype=0, ws=16, n=1 << 30):
    return aq.lib().aq_lora_backward(ad or lora(), dy, ldd, ids, M, s, x, ldx, sx, da, dbt, add, ldadd, dx, lddx, dtype,
                                     ws, n, None)


def test_struct_layout_matches_the_header():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "aq.h")).read(), flags=re.S)
    body = re.search(r"typedef struct aq_lora \{(.*?)\} aq_lora;", src, flags=re.S).group(1)
    fields = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        ptr = "*" in decl
        names = decl.replace("const ", "").split(None, 1)[1]
        fields += [(n.strip(" *"), ptr) for n in names.split(",")]
    assert fields == [(n, t is ctypes.c_void_p) for n, t in aq.AqLoraStruct._fields_]


@pytest.mark.parametrize("kw,status", [
    (dict(ad=lora(a=None)), ARG), (dict(ad=lora(bt=24)), ARG), (dict(ad=lora(off=18)), ARG),
    (dict(ad=lora(scale=None)), ARG), (dict(ad=lora(N=100)), SHAPE), (dict(ad=lora(K=0)), SHAPE),
    (dict(ad=lora(max_rank=257, R=300)), SHAPE), (dict(ad=lora(max_rank=0)), SHAPE), (dict(ad=lora(max_rank=25)), SHAPE),
    (dict(ad=lora(L=0)), SHAPE), (dict(ad=lora(L=16384)), SHAPE), (dict(ad=lora(R=0)), SHAPE),
    (dict(x=None), ARG), (dict(x=24), ARG), (dict(ldx=248), ARG), (dict(ldx=260), ARG), (dict(ids=None), ARG),
    (dict(ids=18), ARG), (dict(M=0), ARG), (dict(M=65535 * 64 + 1), ARG), (dict(y=24), ARG), (dict(ldy=130), ARG),
    (dict(out=None), ARG), (dict(ldo=120), ARG), (dict(dtype=1, ldo=132), ARG), (dict(dtype=2), ARG), (dict(s=18), ARG),
    (dict(ws=None), WORKSPACE), (dict(n=15), WORKSPACE), (dict(M=70, n=64), WORKSPACE), (dict(ws=24), ARG),
    (dict(ldo=132), ARG), (dict(ldo=132, y=32, n=15), WORKSPACE)])  # in place with another pitch, and not in place
def test_lora_apply_refusals(kw, status):
    assert apply(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(ad=lora(bt=None)), ARG), (dict(dy=None), ARG), (dict(dy=24), ARG), (dict(ldd=120), ARG), (dict(ldd=130), ARG),
    (dict(s=None), ARG), (dict(s=18), ARG), (dict(x=None), ARG), (dict(ldx=264), ARG), (dict(sx=None, ldx=260), ARG),
    (dict(sx=18), ARG), (dict(ad=lora(K=248), ldx=256), SHAPE), (dict(da=None), ARG), (dict(dbt=24), ARG),
    (dict(dx=None), ARG), (dict(dx=24), ARG), (dict(lddx=250), ARG), (dict(ldadd=258), ARG), (dict(dtype=7), ARG),
    (dict(M=0), ARG), (dict(ids=None), ARG), (dict(ws=None), WORKSPACE), (dict(n=64), WORKSPACE), (dict(ws=20), ARG),
    (dict(lddx=264), ARG)])
def test_lora_backward_refusals(kw, status):
    assert backward(**kw) == status


M_, N_, K_ = 70, 128, 256
MIB = 1 << 20


def places(**kw):
    """Pointers a MiB apart, some of them moved onto others: 'name' or 'name+bytes'."""
    names = ("x", "ids", "y", "out", "s", "dy", "sx", "da", "dbt", "add", "dx", "ws", "a", "bt", "off", "scale")
    at = {n: (i + 1) * MIB for i, n in enumerate(names)}
    for n, where in kw.items():
        base, _, plus = where.partition("+")
        at[n] = at[base] + int(plus or 0)
    return at


# out over an input, over s, over y a row lower, next to nothing; s over an input
@pytest.mark.parametrize("kw", [
    dict(out="x"), dict(out="x+16"), dict(out="ids"), dict(out="s"), dict(out=f"y+{4 * N_}"), dict(out="y+16"),
    dict(out="a"), dict(out="bt+64"), dict(out="off"), dict(s="x+4"), dict(s="y"), dict(s="ids"), dict(s="scale"),
    dict(x=f"out+{4 * N_ * (M_ - 1)}"), dict(s="y", out="y")])
def test_lora_apply_refuses_overlaps(kw):
    p = places(**kw)
    assert apply(ad=lora(a=p["a"], bt=p["bt"], off=p["off"], scale=p["scale"]), x=p["x"], ids=p["ids"], M=M_, y=p["y"],
                 out=p["out"], s=p["s"], ws=p["ws"]) == ARG


# dx over dy, in place over a residual gradient that is dy itself, over x, and each gradient over what is read or written
@pytest.mark.parametrize("kw", [
    dict(dx="dy"), dict(add="dy", dx="dy"), dict(dy="dx+16"), dict(dx="x"), dict(add="x", dx="x"), dict(dx="x+32"),
    dict(dx="sx"), dict(dx="s"), dict(dx="ids"), dict(dx="add+16"), dict(add=f"dx+{4 * K_}"), dict(dx="a"), dict(dx="bt"),
    dict(da="x"), dict(da="dy+16"), dict(da="s"), dict(da="add"), dict(dbt="dy"), dict(dbt="x+16"), dict(dbt="sx"),
    dict(da="dbt"), dict(da="dx+16"), dict(dbt="dx"), dict(dbt="bt"), dict(da="a"), dict(da="off"), dict(dbt="scale")])
@pytest.mark.parametrize("codes", [True, False])
def test_lora_backward_refuses_overlaps(kw, codes):
    p = places(**kw)
    if not codes and "sx" in kw.values():
        pytest.skip("no token scales")
    assert backward(ad=lora(a=p["a"], bt=p["bt"], off=p["off"], scale=p["scale"]), dy=p["dy"], ids=p["ids"], M=M_,
                    s=p["s"], x=p["x"], sx=p["sx"] if codes else None, da=p["da"], dbt=p["dbt"], add=p["add"],
                    dx=p["dx"], ws=p["ws"]) == ARG


def test_lora_workspace_sizes():
    f = aq.lib().aq_lora_workspace_bytes
    assert f(lora(N=100), 4, 0) == 0 and f(lora(), 0, 0) == 0 and f(None, 4, 0) == 0
    for M in (1, 64, 65, 5000):  # up to 64 tokens take one launch without a workspace
        assert f(lora(), M, 0) == 16 if M <= 64 else f(lora(), M, 0) >= 4 * M * 16
        assert f(lora(), M, 1) >= 4 * M * 16


def gated(gate=16, ldg=256, up=16, ldu=256, M=4, F=256, hq=16, sh=16, gq=16, gs=16, uq=16, us=16):
    return aq.lib().aq_silu_mul_quant(gate, ldg, up, ldu, M, F, hq, sh, gq, gs, uq, us, None)


@pytest.mark.parametrize("kw", [
    dict(gate=None), dict(up=24), dict(hq=24), dict(sh=18), dict(sh=None), dict(gq=None), dict(us=None), dict(gq=24),
    dict(gs=18), dict(M=0), dict(F=8), dict(F=250), dict(F=65552, ldg=65552, ldu=65552), dict(ldg=248), dict(ldu=260)])
def test_gated_refusals(kw):
    assert gated(**kw) == ARG


def gated_back(dh=16, ldd=256, gq=16, gs=16, uq=16, us=16, M=4, F=256, dg=16, ldg=256, du=16, ldu=256):
    return aq.lib().aq_silu_mul_backward(dh, ldd, gq, gs, uq, us, M, F, dg, ldg, du, ldu, None)


@pytest.mark.parametrize("kw", [
    dict(dh=None), dict(dh=24), dict(gq=None), dict(uq=24), dict(gs=18), dict(us=None), dict(M=0), dict(F=24),
    dict(ldd=248), dict(ldg=250), dict(ldu=260), dict(dg=None), dict(du=24)])
def test_gated_backward_refusals(kw):
    assert gated_back(**kw) == ARG


@pytest.mark.parametrize("kw", [
    dict(hq="gate"), dict(hq="up+16"), dict(gq="gate+16"), dict(uq="up"), dict(sh="gate+4"), dict(gs="up"), dict(us="gate"),
    dict(hq="gq"), dict(gq="uq+16"), dict(sh="hq"), dict(gs="us+4"), dict(up="hq+512")])
def test_gated_refuses_overlaps(kw):
    at = {n: (i + 1) * MIB for i, n in enumerate(("gate", "up", "hq", "sh", "gq", "gs", "uq", "us"))}
    for n, where in kw.items():
        at[n] = at[where.split("+")[0]] + int((where.split("+") + ["0"])[1])
    assert gated(M=70, **at) == ARG


@pytest.mark.parametrize("kw", [
    dict(dg="dh+16"), dict(du="dh+16"), dict(du="dh+512"), dict(dg="dh", ldg=264), dict(du="dh", ldu=264),
    dict(dg="dh", du="dh+16"), dict(dg="dh", du="dh"), dict(dg="dh", du="gq"), dict(dg="gq"), dict(du="uq+16"), dict(dg="us"), dict(du="gs"),
    dict(dg="du"), dict(du="dg+16"), dict(dh="dg+35328")])
def test_gated_backward_refuses_overlaps(kw):
    kw = dict(kw)
    at = {n: (i + 1) * MIB for i, n in enumerate(("dh", "gq", "gs", "uq", "us", "dg", "du"))}
    for n in [n for n in kw if n in at]:
        base, _, plus = kw.pop(n).partition("+")
        at[n] = at[base] + int(plus or 0)
    assert gated_back(M=70, **at, **kw) == ARG


def packed(**kw):
    v = dict(N=128, K=256, bN=128, bK=128, R=1, C=2, T4=0, T8=2, bitmap=16, row_off4=16, row_off8=16, tile_idx=16, w4=16,
             w8=16, scales=16)
    v.update(kw)
    return ctypes.byref(aq.AqPackedStruct(**v))


def linear_back(w=None, dy=16, ldd=128, M=4, add=16, ldadd=256, dx=16, lddx=256, dtype=0, ws=16, n=1 << 30):
    return aq.lib().aq_linear_backward(w or packed(), dy, ldd, M, add, ldadd, dx, lddx, dtype, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(w=packed(K=200)), SHAPE), (dict(w=packed(scales=24)), ARG), (dict(w=packed(scale_kind=1)), ARG),
    (dict(dy=None), ARG), (dict(dy=24), ARG), (dict(ldd=120), ARG), (dict(ldd=132), ARG), (dict(M=0), ARG),
    (dict(M=(1 << 21) + 1), ARG), (dict(add=24), ARG), (dict(ldadd=250), ARG), (dict(dx=None), ARG), (dict(dx=8), ARG),
    (dict(lddx=248), ARG), (dict(dtype=1, lddx=260), ARG), (dict(dtype=3), ARG), (dict(ws=None), WORKSPACE),
    (dict(n=16), WORKSPACE), (dict(ws=24), ARG), (dict(lddx=264), ARG)])
def test_linear_backward_refusals(kw, status):
    assert linear_back(**kw) == status


@pytest.mark.parametrize("kw", [
    dict(dx="dy"), dict(add="dy", dx="dy"), dict(dx="dy+16"), dict(dy=f"dx+{4 * 256 * 69}"), dict(dx="add+16"),
    dict(add="dx+1024"), dict(dx="add+64", ldadd=512)])
def test_linear_backward_refuses_overlaps(kw):
    kw = dict(kw)
    at = {n: (i + 1) * MIB for i, n in enumerate(("dy", "add", "dx", "ws"))}
    for n in [n for n in kw if n in at]:
        base, _, plus = kw.pop(n).partition("+")
        at[n] = at[base] + int(plus or 0)
    assert linear_back(M=70, **at, **kw) == ARG


def test_linear_backward_workspace_sizes():
    f = aq.lib().aq_linear_backward_workspace_bytes
    assert f(0, packed()) == 0 and f(4, None) == 0 and f(4, packed(K=200)) == 0
    assert f(4, packed()) >= 256


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        aq.Adapters(torch.zeros(8, 256, dtype=torch.bfloat16), torch.zeros(8, 128, dtype=torch.bfloat16), [8], [1.0])
    with pytest.raises(ValueError):
        aq.aq_silu_mul_quant(x, x)
    with pytest.raises(TypeError):
        aq.aq_silu_mul_quant([[1.0]], x)
    with pytest.raises(ValueError):
        aq.aq_silu_mul_backward(x, x, x, x, x)


@pytest.mark.parametrize("dtype,status", [
    (0x100, WORKSPACE), (0x101, WORKSPACE), (0x200, WORKSPACE), (0x201, WORKSPACE),  # the weights as asked for
    (0x300, ARG), (0x102, ARG), (0x400, ARG), (-1, ARG)])
def test_linear_backward_weights(dtype, status):
    assert linear_back(dtype=dtype, ws=None) == status


@pytest.mark.parametrize("kw", [dict(wait=1000), dict(wait=20_000_000_000), dict(after=-1), dict(kernel=3), dict(kernel=-1),
                                dict(kernel=0, M=64), dict(kernel=1, ad=lora(max_rank=65, R=80)), dict(dx=None)])
def test_stalled_lora_refusals(kw):
    v = dict(ad=lora(), M=70, dx=16, kernel=2, wait=20_000_000, after=0)
    v.update(kw)
    assert aq.lib().aq_debug_lora_backward_stalled(v["ad"], 16, 128, 16, v["M"], 16, 16, 256, 16, 16, 16, v["dx"], 256, 0,
                                                   None, 0, v["kernel"], v["wait"], v["after"], None) == ARG


@pytest.mark.parametrize("wait,after,status", [(1000, 0, ARG), (20_000_000_000, 0, ARG), (20_000_000, -1, ARG),
                                               (20_000_000, 0, WORKSPACE)])
def test_stalled_linear_backward_refusals(wait, after, status):
    assert aq.lib().aq_debug_linear_backward_stalled(packed(), 16, 128, 4, 16, 256, 0, None, 0, wait, after, None) == status
