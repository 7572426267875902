"""norm, add_norm, quantize and scaled_linear without a GPU: the C ABI's argument checks,
plans and workspace sizes, and the binding's refusals.  Nothing is launched."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import scaled_plans as sp
import tiling_roofline_analysis_amd as tra
from tiling_roofline_analysis_amd import norms, scaled

OK, INVALID, UNSUPPORTED = tra.TRA_OK, tra.TRA_ERR_INVALID_ARG, tra.TRA_ERR_UNSUPPORTED
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# addresses that are never read
X, H, W, B, G, PW, PB, R, Y, DR, DY, DX, DH, DW, DB, DG, DPW, DPB, WS = (
    i << 40 for i in range(1, 20))
FAR = 1 << 47


def test_packed_structs_match_the_header(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    names = (("tra_norm_args", "Y"), ("tra_norm_grad_args", "workspace"),
             ("tra_quantize_args", "ST"), ("tra_scaled_args", "workspace"))
    src = tmp_path / "s.c"
    src.write_text('#include "tra_gemm.h"\n#include <stdio.h>\n#include <stddef.h>\nint main(void){'
                   + "".join(f'printf("%zu %zu ",sizeof({t}),offsetof({t},{f}));' for t, f in names)
                   + "return 0;}\n")
    exe = tmp_path / "s"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = list(map(int, subprocess.run([str(exe)], capture_output=True, text=True,
                                       check=True).stdout.split()))
    sizes = [s.size for s in (norms._ARGS, norms._GRAD_ARGS, scaled._QUANTIZE, scaled._SCALED)]
    assert got[0::2] == sizes
    # the last pointer's place: behind it a leading dimension, a size, two strides, a size
    assert got[1::2] == [sizes[0] - 16, sizes[1] - 16, sizes[2] - 24, sizes[3] - 16]


# --- norms ------------------------------------------------------------------------------

FWD = ("dtype pdtype norm post M D groups scale eps X ldx H ldh weight bias gate post_weight "
       "post_bias ldw ldb ldg ldpw ldpb R ldr Y ldy").split()
BWD = FWD[:-4] + "dR lddr dY lddy dX lddx dH lddh dw db dg dpw dpb ws ws_bytes".split()


def fwd(**kw):
    a = dict(dtype=1, pdtype=1, norm=1, post=1, M=8, D=64, groups=1, scale=1.0, eps=1e-6, X=X,
             ldx=64, H=H, ldh=64, weight=W, bias=B, gate=G, post_weight=PW, post_bias=PB, ldw=0,
             ldb=0, ldg=0, ldpw=0, ldpb=0, R=R, ldr=64, Y=Y, ldy=64)
    assert set(kw) <= set(a)
    a.update(kw)
    return norms._ARGS.pack(*(a[k] for k in FWD))


def bwd(**kw):
    a = dict(dtype=1, pdtype=1, norm=1, post=1, M=8, D=64, groups=1, scale=1.0, eps=1e-6, X=X,
             ldx=64, H=H, ldh=64, weight=W, bias=B, gate=G, post_weight=PW, post_bias=PB, ldw=0,
             ldb=0, ldg=0, ldpw=0, ldpb=0, dR=DR, lddr=64, dY=DY, lddy=64, dX=DX, lddx=64, dH=DH,
             lddh=64, dw=DW, db=DB, dg=DG, dpw=DPW, dpb=DPB, ws=WS, ws_bytes=FAR)
    assert set(kw) <= set(a)
    a.update(kw)
    return norms._GRAD_ARGS.pack(*(a[k] for k in BWD))


def norm(**kw):
    return tra.load().tra_norm(fwd(**kw), None)


def grad_size(**kw):
    n = ctypes.c_size_t(0)
    return tra.load().tra_norm_backward_workspace_size(bwd(**kw), ctypes.byref(n)), n.value


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=-1), dict(pdtype=2), dict(dtype=0, pdtype=1), dict(norm=3),
    dict(norm=-1), dict(post=3), dict(M=-1), dict(D=-1), dict(groups=0), dict(groups=3),
    dict(eps=-1.0), dict(eps=float("nan")), dict(X=0), dict(Y=0), dict(ldx=63), dict(ldh=63),
    dict(ldy=63), dict(ldr=63), dict(X=X + 1), dict(weight=W + 1),
    dict(H=0), dict(H=0, post=0, post_weight=0, post_bias=0),               # a gate, R without H
    dict(post=0), dict(norm=0), dict(norm=0, weight=0, bias=0),              # vectors, Y of none
    dict(norm=0, weight=0, bias=0, Y=0, R=0),                               # nothing to write
    dict(ldw=63, groups=2), dict(Y=X), dict(Y=X + 2), dict(Y=R), dict(R=H), dict(R=X + 128),
    dict(Y=W), dict(R=G)])
def test_norm_refuses(bad):
    assert norm(**bad) == INVALID


def test_norm_limits_and_empty_matrices():
    assert norm(M=(1 << 30) + 2, groups=2) == UNSUPPORTED
    assert norm(D=(1 << 30) + 1) == UNSUPPORTED
    assert norm(M=70000 * 2, groups=70000) == UNSUPPORTED
    for empty in (dict(M=0), dict(D=0)):
        assert norm(X=0, H=0, R=0, Y=0, **empty) == OK
    assert tra.load().tra_norm(None, None) == INVALID


@pytest.mark.parametrize("bad", [
    dict(dtype=7), dict(pdtype=0, dtype=2, weight=W + 2), dict(groups=3), dict(X=0), dict(lddr=1),
    dict(lddy=1), dict(H=0), dict(H=0, post=0, gate=0, post_weight=0, post_bias=0, dH=0, dpw=0,
                                  dpb=0, dg=0),                             # dR without H
    dict(norm=0, weight=0, dw=0, db=0), dict(norm=0, weight=0, dY=0, dw=0),
    dict(weight=0), dict(gate=0), dict(post_weight=0), dict(post=0, post_weight=0, dpw=0),
    dict(dX=DR), dict(dX=DY), dict(dX=X), dict(dH=H), dict(dH=DX), dict(dw=W), dict(dg=DX),
    dict(dw=DB), dict(dX=DX + 1)])
def test_norm_backward_refuses(bad):
    assert tra.load().tra_norm_backward(bwd(**bad), None) == INVALID
    assert grad_size(**bad)[0] == INVALID


def test_norm_backward_checks_its_workspace():
    st, need = grad_size()
    assert st == OK and need > 0
    for ws, size in ((0, need), (WS, need - 1), (WS + 128, need)):
        assert tra.load().tra_norm_backward(bwd(ws=ws, ws_bytes=size), None) == INVALID
    assert grad_size(dw=0, db=0, dg=0, dpw=0, dpb=0) == (OK, 0)
    # sums of a row for each of some chunks; wide rows keep statistics too
    st, small = grad_size(M=512, db=0, dg=0, dpw=0, dpb=0)
    assert st == OK and small <= 512 * 64 * 4
    st, wide = grad_size(M=512, D=9000, ldx=9000, ldh=9000, lddr=9000, lddy=9000, lddx=9000,
                         lddh=9000)
    # (statistics, and five sums of some 2 to 512 chunks of rows)
    assert st == OK and 5 * 2 * 9000 * 4 <= wide - 512 * 8 * 4 <= 5 * 512 * 9000 * 4
    n = ctypes.c_size_t(0)
    assert tra.load().tra_norm_backward_workspace_size(None, ctypes.byref(n)) == INVALID
    assert tra.load().tra_norm_backward_workspace_size(bwd(), None) == INVALID


# --- quantize ------------------------------------------------------------------------------

QUANT = "dtype fp8 scale rows M K X ldx Q ldq S ss_row ss_block QT ldqt ST sts_row sts_block".split()


def quant(**kw):
    a = dict(dtype=1, fp8=0, scale=1, rows=1, M=200, K=300, X=X, ldx=300, Q=H, ldq=304, S=W,
             ss_row=1, ss_block=200, QT=B, ldqt=208, ST=G, sts_row=1, sts_block=300)
    assert set(kw) <= set(a)
    a.update(kw)
    return tra.load().tra_quantize(scaled._QUANTIZE.pack(*(a[k] for k in QUANT)), None)


@pytest.mark.parametrize("bad", [
    dict(dtype=5), dict(fp8=2), dict(fp8=-1), dict(scale=2), dict(rows=64), dict(rows=0),
    dict(M=-1), dict(K=-1), dict(X=0), dict(ldx=299), dict(X=X + 1), dict(Q=0, QT=0), dict(S=0),
    dict(ST=0), dict(ldq=300), dict(ldq=303), dict(ldq=312), dict(Q=H + 8), dict(ldqt=200),
    dict(ldqt=216), dict(ss_row=2, ss_block=2), dict(ss_row=0), dict(ss_block=199),
    dict(ss_row=2, ss_block=1), dict(sts_block=299), dict(scale=0, S=W + 2), dict(Q=X),
    dict(S=X), dict(QT=H), dict(ST=W), dict(S=H), dict(Q=X + 64)])
def test_quantize_refuses(bad):
    assert quant(**bad) == INVALID


def test_quantize_limits_and_empty_matrices():
    assert quant(M=(1 << 30) + 1) == UNSUPPORTED
    assert quant(M=1 << 29, K=1 << 20, ldx=1 << 20) == UNSUPPORTED
    assert quant(M=0, X=0, Q=0, QT=0) == OK and quant(K=0, X=0, Q=0, QT=0) == OK
    assert tra.load().tra_quantize(None, None) == INVALID


# --- scaled_linear ----------------------------------------------------------------------

def product(**kw):
    return tra.load().tra_scaled_linear(sp.pack(**kw), None)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(x_dtype=3), dict(x_dtype=-2), dict(x_fp8=2), dict(w_fp8=2), dict(scale=2),
    dict(w_block_rows=2), dict(M=-1), dict(N=-1), dict(K=-1), dict(X=0), dict(W=0), dict(SX=0),
    dict(SW=0), dict(Y=0), dict(ldx=255), dict(ldw=240), dict(ldw=264), dict(X=sp.X + 8),
    dict(W=sp.W + 4), dict(ldy=63), dict(R=sp.R, ldr=63), dict(sx_row=2, sx_block=2),
    dict(scale=0, w_block_rows=1), dict(x_fp8=1, w_fp8=1), dict(w_fp8=1, scale=0),
    dict(w_fp8=1, x_dtype=1), dict(Y=sp.X), dict(Y=sp.W), dict(Y=sp.SX), dict(Y=sp.SW),
    dict(bias=sp.Y), dict(R=sp.Y + 2, ldr=64), dict(R=sp.Y, ldr=128), dict(Y=sp.Y + 1)])
def test_scaled_linear_refuses(bad):
    assert product(**bad) == INVALID


def test_scaled_linear_limits_and_empty_matrices():
    assert product(M=(1 << 30) + 1) == UNSUPPORTED
    assert product(K=1 << 22) == UNSUPPORTED
    assert product(ldw=1 << 22) == UNSUPPORTED
    assert product(ldx=1 << 22) == UNSUPPORTED
    assert product(sx_row=1 << 22, sx_block=1) == UNSUPPORTED
    assert product(M=300, N=300, w_block_rows=1, sw_row=1 << 22) == UNSUPPORTED
    assert product(M=1 << 28, N=1 << 28, ldy=1 << 28, sx_block=1 << 28) == UNSUPPORTED
    assert product(M=0) == OK and product(N=0, ldy=0) == OK
    assert tra.load().tra_scaled_linear(None, None) == INVALID


def size(**kw):
    n = ctypes.c_size_t(0)
    st = tra.load().tra_scaled_linear_workspace_size(sp.pack(**kw), ctypes.byref(n))
    return st, n.value


def test_scaled_linear_checks_its_workspace():
    # a quantized copy of x, and the sums of a split
    call = dict(M=64, N=64, K=4096)
    st, given = size(**call)
    st2, made = size(**call, x_dtype=1)
    assert st == st2 == OK and given > 0 and made >= given + 64 * 4096 + 64 * 32
    for ws, have in ((0, given), (sp.WS, given - 1), (sp.WS + 16, given)):
        assert product(**call, ws=ws, ws_bytes=have) == INVALID
    assert size(M=1, N=64, K=256, x_dtype=1) == (OK, 0)


@pytest.mark.parametrize("scale,dtype,block_rows", [
    ("e8m0", 1, 128), ("e8m0", 1, 1), ("f32", 1, 128), ("e8m0", 0, 128), ("e8m0", 0, 1),
    ("f32", 0, 128)])
def test_plans_reach_every_kernel(scale, dtype, block_rows):
    seen = {sp.reached(*c, scale, dtype=dtype, w_block_rows=block_rows) for c in sp.CALLS}
    # binary32 results with a scale for each row of the weights have no 128 x 128
    tiles = ["64x64", "64x128"] + (["128x128"] if dtype or block_rows == 128 else [])
    want = {("scaled_tile", t, deep) for t in tiles for deep in (0, 1)} | {("scaled_few", "16x16", 0)}
    want |= {("scaled_wide", "256x256", 0)} if dtype else set()
    assert {s[:3] for s in seen} == want
    splits = {(t, s) for k, t, _, s in seen if k == "scaled_tile"}
    assert splits >= {(t, s) for t in tiles for s in ("no", "all", "last")}
    if dtype:
        assert {s for k, _, _, s in seen if k == "scaled_wide"} == {"no", "last"}


@pytest.mark.parametrize("scale", ["e8m0", "f32"])
def test_plans_for_few_rows(scale):
    made = {d["quantizes"] for c in sp.CALLS for d in [dict(kv.split("=") for kv in sp.describe(
        *c, scale, x_dtype=1).split())] if d["kernel"] == "scaled_few"}
    assert made == {"1", "2"}


def test_describe_into_small_buffers():
    for n in (1, 2, 20, 60, 400):
        buf = ctypes.create_string_buffer(b"x" * 500, 500)
        assert tra.load().tra_scaled_linear_describe(sp.pack(), buf, n) == OK
        assert 0 in buf.raw[:n] and buf.raw[n:n + 1] == b"x"
    assert tra.load().tra_scaled_linear_describe(sp.pack(), None, 0) == OK
    assert tra.load().tra_scaled_linear_describe(sp.pack(), None, 4) == INVALID
    buf = ctypes.create_string_buffer(400)
    assert tra.load().tra_scaled_linear_describe(sp.pack(M=0), buf, 400) == OK
    assert buf.value == b"kernel=none"


# --- the binding -------------------------------------------------------------------------

def test_operators_are_there_by_name():
    for name in ("norm", "add_norm", "norm_backward", "add_norm_backward", "quantize",
                 "scaled_linear", "scaled_linear_backward"):
        assert callable(getattr(tra, name)) and getattr(tra, name).__doc__


def test_tensors_on_the_host_are_refused():
    x = torch.ones(4, 32)
    w = x.to(torch.float8_e4m3fn)
    for call in (lambda: tra.norm(x), lambda: tra.add_norm(x, x), lambda: tra.quantize(x),
                 lambda: tra.scaled_linear(x, x.t()), lambda: tra.scaled_linear(x, w.t()),
                 lambda: tra.norm_backward(x, x), lambda: tra.add_norm_backward(x, x, x, x),
                 lambda: tra.scaled_linear_backward(x, x, x.t()), lambda: tra.norm(None),
                 lambda: tra.quantize([1.0]), lambda: tra.scaled_linear(None, x),
                 lambda: tra.add_norm(x, None)):
        with pytest.raises(TypeError):
            call()


def test_names_of_kinds_and_forms():
    x = torch.ones(4, 32)
    for call in (lambda: tra.norm(x, kind="none"), lambda: tra.norm(x, kind=None),
                 lambda: tra.add_norm(x, x, kind="l2"), lambda: tra.add_norm(x, x, post=["rms"]),
                 lambda: tra.add_norm(x, x, kind="none", weight=x[0]),
                 lambda: tra.add_norm(x, x, post_bias=x[0]),
                 lambda: tra.quantize(x, block=64), lambda: tra.quantize(x, form="all"),
                 lambda: tra.quantize(x, dtype=torch.int8),
                 lambda: tra.quantize(x, scale_dtype=torch.float64)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        tra.norm(x, eps=x[0, 0])


CALLS = {"norm": lambda t: tra.norm(t), "add_norm": lambda t: tra.add_norm(t, t)[1],
         "quantize": lambda t: tra.quantize(t)[0],
         "scaled_linear": lambda t: tra.scaled_linear(t, t.t())}


@pytest.mark.parametrize("name", list(CALLS))
def test_what_would_lose_the_call_is_refused(name):
    from torch.autograd import forward_ad
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(torch.ones(2, 32), torch.ones(2, 32))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            CALLS[name](dual)
    with pytest.raises(RuntimeError, match="jit.trace"):
        torch.jit.trace(CALLS[name], torch.ones(2, 32))
