"""Products of 8-bit matrices that reach every kernel and way of splitting it."""
from __future__ import annotations

import ctypes

import tiling_roofline_analysis_amd as tra
from tiling_roofline_analysis_amd import scaled

# (M, N, K): few rows, quantized by the kernel and before it; then the tiles (found by a
# search of 60000 random products, the cheapest that reach them all)
CALLS = [(1, 16, 128), (1, 500, 4096), (3, 48, 9000), (16, 1030, 272), (9, 33, 16),
         (2, 4100, 1300), (19, 9, 16), (18, 9, 2069), (73, 8900, 17), (6878, 264, 16),
         (816, 5074, 268), (680, 1513, 3341), (1135, 273, 7425), (2944, 66, 3777),
         (2527, 1619, 1986), (1233, 777, 6251), (796, 1382, 6786), (2604, 4666, 736),
         (1977, 1462, 4526), (7203, 2255, 640), (1675, 1250, 10057), (69, 4183, 8929),
         (7356, 2239, 2451), (7177, 1736, 16), (763, 2792, 1140), (2695, 386, 5244),
         (2735, 75, 2875)]

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


def reached(M, N, K, scale, **kw):
    """(kernel, tile, deep, split) of a call: split is no, all tiles, or the last ones."""
    d = dict(kv.split("=") for kv in describe(M, N, K, scale, **kw).split())
    split = "no" if d["splits"] == "1" else "all" if d["whole"] == "0" else "last"
    return d["kernel"], d["tile"], int(d["deep"]) if d["kernel"] == "scaled_tile" else 0, split
