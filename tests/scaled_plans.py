"""Products of 8-bit matrices that reach every kernel and way of splitting it."""
from __future__ import annotations

import ctypes

import tiling_roofline_analysis_amd as tra
from tiling_roofline_analysis_amd import scaled

# (M, N, K)
CALLS = [(1, 16, 128), (1, 500, 4096), (3, 48, 9000), (16, 1030, 272), (9, 33, 16), (2, 4100, 1300), (40, 60, 500), (64, 64, 4096), (130, 520, 264), (300, 700, 1040),
         (515, 1030, 520), (1000, 1100, 144), (1500, 2000, 300), (2100, 4100, 136),
         (70, 4100, 6000), (4100, 4200, 400), (1030, 4100, 2064)]

# addresses that are never read
X, SX, W, SW, BIAS, R, Y, WS = (i << 40 for i in range(1, 9))


def pack(M=8, N=64, K=256, **kw):
    a = dict(dtype=1, x_dtype=-1, x_fp8=0, w_fp8=0, scale=1, w_block_rows=128, M=M, N=N, K=K, X=X,
             ldx=-(-K // 16) * 16, SX=SX, sx_row=1, sx_block=M, W=W, ldw=-(-K // 16) * 16, SW=SW,
             sw_row=-(-K // 128), sw_block=1, bias=0, R=0, ldr=0, Y=Y, ldy=N, ws=0, ws_bytes=0)
    a.update(kw)
    return scaled._SCALED.pack(*a.values())


def describe(M, N, K, scale, **kw) -> str:
    buf = ctypes.create_string_buffer(512)
    st = tra.load().tra_scaled_linear_describe(
        pack(M, N, K, scale=1 if scale == "e8m0" else 0, **kw), buf, len(buf))
    assert st == tra.TRA_OK, st
    return buf.value.decode()
