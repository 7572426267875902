"""The fused linear operators' C ABI and binding without a GPU: names, argument
checks, plans and workspace sizes.  Nothing is launched."""
from __future__ import annotations

import ctypes

import pytest
import torch

import tiling_roofline_analysis_amd as tra
from tiling_roofline_analysis_amd import fused

OK, INVALID, UNSUPPORTED = tra.TRA_OK, tra.TRA_ERR_INVALID_ARG, tra.TRA_ERR_UNSUPPORTED
FWD = ("dtype act w_trans gated M N K X ldx W W2 ldw bias R ldr Y ldy Z ldz ws ws_bytes").split()
BWD = ("dtype act w_trans gated M N K dY lddy Z ldz X ldx W W2 ldw dX lddx dW dW2 lddw dbias "
       "ws ws_bytes").split()
# addresses that are never read: every call here is answered on the host
X, W, W2, BIAS, R, Y, Z, DY, DX, DW, DW2, DB, WS = (i << 40 for i in range(1, 14))


def fwd(**kw):
    a = dict(dtype=1, act=0, w_trans=0, gated=0, M=8, N=64, K=32, X=X, ldx=32, W=W, W2=0,
             ldw=64, bias=0, R=0, ldr=0, Y=Y, ldy=64, Z=0, ldz=0, ws=0, ws_bytes=0)
    a.update(kw)
    return fused._ARGS.pack(*(a[k] for k in FWD))


def bwd(**kw):
    a = dict(dtype=1, act=4, w_trans=0, gated=0, M=8, N=64, K=32, dY=DY, lddy=64, Z=Z, ldz=64,
             X=X, ldx=32, W=W, W2=0, ldw=64, dX=DX, lddx=32, dW=DW, dW2=0, lddw=64, dbias=0, ws=0,
             ws_bytes=0)
    a.update(kw)
    return fused._GRAD_ARGS.pack(*(a[k] for k in BWD))


def size(packed, name="tra_linear_workspace_size"):
    n = ctypes.c_size_t(0)
    st = getattr(tra.load(), name)(packed, ctypes.byref(n))
    return st, n.value


def bsize(packed):
    return size(packed, "tra_linear_backward_workspace_size")


def test_packed_structs_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "s.c"
    src.write_text('#include "tra_gemm.h"\n#include <stdio.h>\n#include <stddef.h>\n'
                   "int main(void){printf(\"%zu %zu %zu %zu %zu %zu\\n\","
                   "sizeof(tra_linear_args),offsetof(tra_linear_args,Y),"
                   "offsetof(tra_linear_args,workspace),sizeof(tra_linear_grad_args),"
                   "offsetof(tra_linear_grad_args,dX),"
                   "offsetof(tra_linear_grad_args,workspace));return 0;}\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "s")
    subprocess.run([cc, "-I", os.path.join(root, "include"), str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True,
                                          check=True).stdout.split()]

    def offset(fmt, fields, field):
        # the offset where a marker in that field lands
        raw = fmt.pack(*[0x7e if f == field else 0 for f in fields])
        return raw.index(0x7e)

    assert got == [fused._ARGS.size, offset(fused._ARGS, FWD, "Y"),
                   offset(fused._ARGS, FWD, "ws"), fused._GRAD_ARGS.size,
                   offset(fused._GRAD_ARGS, BWD, "dX"), offset(fused._GRAD_ARGS, BWD, "ws")]


@pytest.mark.parametrize("bad", [
    dict(dtype=-1), dict(dtype=3), dict(act=-1), dict(act=6), dict(w_trans=2), dict(gated=2),
    dict(M=-1), dict(N=-1), dict(K=-1), dict(X=0), dict(W=0), dict(Y=0), dict(ldx=31),
    dict(ldw=63), dict(ldy=63), dict(w_trans=1, ldw=31), dict(R=R, ldr=63), dict(Z=Z, ldz=63),
    dict(X=X + 1), dict(Y=Y + 1), dict(Z=Z + 2, ldz=64), dict(bias=BIAS + 1), dict(W2=W2),
    dict(Y=X), dict(Y=W), dict(Y=X + 16), dict(bias=Y), dict(R=Y + 2, ldr=64),
    dict(R=Y, ldr=65), dict(Z=Y, ldz=64), dict(Z=X, ldz=64), dict(Y=W + 62 * 2, ldy=64),
    dict(X=(1 << 64) - 64), dict(ldx=1 << 62),
], ids=str)
def test_linear_refuses(bad):
    assert tra.load().tra_linear(fwd(**bad), None) == INVALID
    assert size(fwd(**bad))[0] == INVALID


@pytest.mark.parametrize("bad", [
    dict(W2=0), dict(bias=BIAS), dict(R=R, ldr=64), dict(Z=Z, ldz=127), dict(Y=W2),
    dict(W2=W2 + 1),
], ids=str)
def test_gated_linear_refuses(bad):
    assert tra.load().tra_linear(fwd(**{"gated": 1, "W2": W2, **bad}), None) == INVALID


@pytest.mark.parametrize("bad", [
    dict(dtype=9), dict(act=17), dict(w_trans=-1), dict(gated=-1), dict(K=-5), dict(dY=0),
    dict(Z=0), dict(X=0), dict(W=0), dict(lddy=63), dict(ldz=63), dict(lddx=31), dict(lddw=63),
    dict(dX=DY), dict(dX=X), dict(dW=W), dict(dW=DX), dict(dbias=DX), dict(dbias=DB + 1),
    dict(W2=W2), dict(dW2=DW2), dict(dX=DX + 1),
], ids=str)
def test_linear_backward_refuses(bad):
    assert tra.load().tra_linear_backward(bwd(**bad), None) == INVALID


@pytest.mark.parametrize("bad", [
    dict(W2=0), dict(dW2=0), dict(dW=0), dict(dbias=DB), dict(Z=0), dict(ldz=127), dict(dW2=DW),
], ids=str)
def test_gated_backward_refuses(bad):
    a = dict(gated=1, W2=W2, dW2=DW2, ldz=128)
    a.update(bad)
    assert tra.load().tra_linear_backward(bwd(**a), None) == INVALID


def test_null_arguments():
    lib = tra.load()
    assert lib.tra_linear(None, None) == INVALID
    assert lib.tra_linear_backward(None, None) == INVALID
    assert size(None)[0] == INVALID and bsize(None)[0] == INVALID
    assert lib.tra_linear_workspace_size(fwd(), None) == INVALID
    assert lib.tra_linear_describe(None, None, 0) == INVALID


def test_sizes_past_the_limits_are_unsupported():
    big = 1 << 31
    assert tra.load().tra_linear(fwd(M=big), None) == UNSUPPORTED
    assert tra.load().tra_linear(fwd(M=1 << 29, N=1 << 29, ldw=1 << 29, ldy=1 << 29, W=1 << 58,
                                     Y=1 << 61), None) == UNSUPPORTED
    assert tra.load().tra_linear_backward(bwd(K=big, ldx=big, lddx=big), None) == UNSUPPORTED
    # rows that a weight gradient sums over, within a tile of 32 bits
    rows = (1 << 31) - 8
    assert tra.load().tra_linear_backward(bwd(M=rows, dX=0), None) == UNSUPPORTED
    wide = 1 << 28
    assert tra.load().tra_linear_backward(
        bwd(N=wide, K=1, lddy=wide, ldz=wide, ldw=wide, lddw=wide, ldx=1, lddx=1, dbias=DB),
        None) == UNSUPPORTED


def test_empty_results_need_nothing():
    assert tra.load().tra_linear(fwd(M=0, X=0, Y=0), None) == OK
    assert tra.load().tra_linear(fwd(N=0, W=0, Y=0), None) == OK
    assert tra.load().tra_linear(fwd(M=0, X=0, Y=0, W2=W2, gated=1), None) == OK
    assert tra.load().tra_linear_backward(bwd(M=0, K=0, dY=0, Z=0), None) == OK


def test_column_ranges_of_one_buffer_do_not_overlap():
    # Y, N = 64 wide, behind X, 32 wide, in rows of 96
    assert size(fwd(ldx=96, Y=X + 64, ldy=96))[0] == OK
    assert size(fwd(ldx=96, Y=X + 62, ldy=96))[0] == INVALID
    # the halves of a packed weight gradient
    a = dict(gated=1, W2=W2, ldz=128, dW2=DW + 128, lddw=128)
    assert bsize(bwd(**a))[0] == OK
    assert bsize(bwd(**{**a, "dW2": DW + 126}))[0] == INVALID
    # the residual in place
    assert size(fwd(R=Y, ldr=64))[0] == OK


@pytest.mark.parametrize("shape", [(1, 1, 1), (5, 7, 9), (16, 4096, 12288), (333, 8192, 2048),
                                   (37, 5461, 2048), (100, 100, 100000), (4096, 64, 4096)])
@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_workspace_is_checked(shape, dtype):
    M, N, K = shape
    a = dict(dtype=dtype, M=M, N=N, K=K, ldx=K, ldw=N, ldy=N)
    st, need = size(fwd(**a))
    assert st == OK
    if need:
        lib = tra.load()
        assert lib.tra_linear(fwd(**a), None) == INVALID
        assert lib.tra_linear(fwd(**a, ws=WS, ws_bytes=need - 1), None) == INVALID
        assert lib.tra_linear(fwd(**a, ws=WS + 16, ws_bytes=need), None) == INVALID
    b = dict(dtype=dtype, M=M, N=N, K=K, ldx=K, ldw=N, lddy=N, ldz=N, lddx=K, lddw=N, dbias=DB)
    st, need = bsize(bwd(**b))
    # dZ itself and the column sums at least
    assert st == OK and need >= M * N * (4 if dtype == 0 else 2) + 4 * N
    assert tra.load().tra_linear_backward(bwd(**b, ws=WS, ws_bytes=need - 1), None) == INVALID


def describe(packed):
    buf = ctypes.create_string_buffer(256)
    assert tra.load().tra_linear_describe(packed, buf, 256) == OK
    return dict(kv.split("=") for kv in buf.value.decode().split())


def test_describe_tells_aligned_from_unaligned():
    a = dict(M=512, N=512, K=512, ldx=512, ldw=512, ldy=512)
    assert describe(fwd(**a))["loads"] == "direct"
    assert describe(fwd(**{**a, "ldx": 513}))["loads"] == "registers"
    assert describe(fwd(**{**a, "X": X + 2}))["loads"] == "registers"
    assert describe(fwd(**{**a, "N": 511}))["loads"] == "registers"
    assert describe(fwd(M=0, X=0, Y=0)) == {"kernel": "none"}


def plan(M, N, K, dtype, layout, gated=0, pad=0):
    kn = layout == "kn"
    return describe(fwd(M=M, N=N, K=K, dtype=dtype, w_trans=0 if kn else 1, gated=gated,
                        W2=W2 if gated else 0, ldx=K + pad, ldw=(N if kn else K) + pad, ldy=N))


@pytest.mark.parametrize("args, want", [
    # one token: straight from memory; few strips and a long K: a split instead
    ((1, 2048, 2048, 1, "nk"), dict(kernel="linear_few", splits="1")),
    ((16, 1024, 1024, 0, "kn"), dict(kernel="linear_few", tile="16x16")),
    ((1, 12288, 4096, 1, "nk", 1), dict(kernel="linear_few", tile="16x32")),
    ((2, 512, 8192, 1, "kn"), dict(kernel="linear_tile")),
    # many 16-bit tiles
    ((8192, 12288, 4096, 1, "nk", 1), dict(tile="256x256", loads="direct")),
    ((4096, 4096, 4096, 2, "kn"), dict(tile="256x256")),
    # ... not in binary32, nor unaligned
    ((4096, 4096, 4096, 0, "kn"), dict(tile="128x128", loads="direct")),
    ((4096, 4096, 4096, 1, "kn", 0, 1), dict(tile="128x128", loads="registers")),
    ((4096, 4096, 4096, 0, "nk", 0, 1), dict(tile="64x128", loads="direct")),
    # a tile a CU
    ((1024, 1024, 1024, 0, "kn"), dict(tile="64x64", splits="1")),
    ((333, 8192, 2048, 1, "nk"), dict(tile="128x128", splits="1")),
], ids=str)
def test_plans(args, want):
    got = plan(*args)
    assert {k: got[k] for k in want} == want, got


def test_splits_cover_every_k_tile_once():
    for M, N, K, dtype in ((20, 200, 100000, 1), (100, 500, 7777, 0), (64, 64, 64, 2),
                           (17, 1000, 12345, 2), (300, 300, 30000, 0), (3000, 2049, 1531, 0),
                           (4200, 4200, 4096, 1), (4608, 4608, 4096, 2)):
        d = plan(M, N, K, dtype, "nk")
        tiles = -(-K // (32 if dtype == 0 else 64))
        splits = int(d["splits"])
        per = -(-tiles // splits)
        assert (splits - 1) * per < tiles <= splits * per
        bm, bn = (int(v) for v in d["tile"].split("x"))
        split_tiles = -(-M // bm) * -(-N // bn) - int(d["whole"])
        assert (split_tiles > 0) == (splits > 1)
        assert int(d["workspace_bytes"]) == (splits > 1) * split_tiles * splits * bm * bn * 4


def test_binding_refuses_cpu_tensors_and_bad_arguments():
    x, w = torch.ones(2, 3), torch.ones(3, 4)
    with pytest.raises(TypeError):
        tra.linear(x, w)
    with pytest.raises(TypeError):
        tra.gated_linear(x, w, w)
    with pytest.raises(TypeError):
        tra.linear([1.0], w)
    with pytest.raises(TypeError):
        tra.gated_linear(x, w, None)
    with pytest.raises(ValueError):
        tra.linear(x, w, act="swish")
    with pytest.raises(ValueError):
        tra.linear(x, w, act=None)


def test_unknown_names_still_raise():
    with pytest.raises(AttributeError):
        tra.no_such_operator


@pytest.mark.parametrize("bad", [
    dict(X=Y), dict(W=Y), dict(bias=Y), dict(w_trans=1, W=Y), dict(M=1, X=Y), dict(M=1, bias=Y),
], ids=str)
def test_only_the_residual_may_be_the_result(bad):
    # the residual in place, and another operand at the same address with it
    a = dict(N=32, ldw=32, ldy=32, R=Y, ldr=32)
    assert size(fwd(**a))[0] == OK
    assert size(fwd(**{**a, **bad}))[0] == INVALID
    assert tra.load().tra_linear(fwd(**{**a, **bad}), None) == INVALID


CALLS = {"linear": lambda t: tra.linear(t, torch.ones(3, 4)),
         "gated_linear": lambda t: tra.gated_linear(torch.ones(2, 3), t, torch.ones(3, 4)),
         "linear_backward": lambda t: tra.linear_backward(t, torch.ones(2, 3), torch.ones(3, 4)),
         "gated_linear_backward": lambda t: tra.gated_linear_backward(
             torch.ones(2, 4), torch.ones(2, 3), t, torch.ones(3, 4), torch.ones(2, 8))}


@pytest.mark.parametrize("name", list(CALLS))
def test_forward_mode_derivatives_are_refused(name):
    # (before anything else is looked at, so also for tensors on the CPU)
    from torch.autograd import forward_ad
    call = CALLS[name]
    with forward_ad.dual_level():
        t = torch.ones(2, 3)
        with pytest.raises(NotImplementedError, match="forward-mode"):
            call(forward_ad.make_dual(t, t))
        with torch.no_grad(), pytest.raises(NotImplementedError, match="forward-mode"):
            call(forward_ad.make_dual(t, t))
        with pytest.raises(TypeError):
            call(t)                      # no tangent: the other checks answer
    with pytest.raises(TypeError):
        call(t)


@pytest.mark.parametrize("name", list(CALLS))
def test_tracing_is_refused(name):
    with pytest.raises(RuntimeError, match="jit.trace"):
        torch.jit.trace(CALLS[name], torch.ones(2, 3))


def test_a_kept_tensor_that_requires_a_gradient_is_refused():
    # overwriting it would leave autograd with the gradient of what it was
    x, w = torch.ones(2, 3), torch.ones(3, 4)
    z = torch.empty(2, 8, requires_grad=True)
    with pytest.raises(ValueError, match="out and z"):
        tra.linear(x, w, z=z[:, :4])
    with pytest.raises(ValueError, match="out and z"):
        tra.gated_linear(x, w, w, z=z)
    with torch.no_grad(), pytest.raises(TypeError):
        tra.linear(x, w, z=z[:, :4])         # nothing is recorded: the other checks answer


def test_plans_do_not_depend_on_what_is_kept():
    # so that a result has the same bits with and without gradients
    import math
    import random
    rng = random.Random(5)

    def size(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi))))

    for _ in range(600):
        M, N, K = size(1, 8192), size(64, 12288), size(64, 12288)
        if rng.random() < 0.7:
            N, K = -(-N // 8) * 8, -(-K // 8) * 8
        nk, gated = rng.choice([0, 1]), rng.choice([0, 1])
        a = dict(M=M, N=N, K=K, dtype=rng.choice([0, 1, 2]), w_trans=nk, gated=gated,
                 W=1 << 50, W2=1 << 51 if gated else 0, ldx=K, ldw=K if nk else N, ldy=N)
        want = describe(fwd(**a))
        assert describe(fwd(**a, Z=1 << 60, ldz=N * (1 + gated))) == want, a
        if not gated:
            assert describe(fwd(**a, bias=1 << 52, R=1 << 53, ldr=N, act=4)) == want, a
