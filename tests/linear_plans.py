"""Calls of the fused linear operators that between them launch every kernel instance
with every way of splitting it that a call can reach.

A row is a forward call and both products of its backward call: sizes, type, layout
of the weights, gated or not, elements of padding behind each row, and whether rows
lie 4 MB apart.  The plans that a row leads to are the library's own choice, so a
change of the planner's constants moves them: test_linear_plans_cpu.py then says what
is no longer covered, and

    python tests/linear_plans.py [SECONDS]

searches random calls for rows that cover everything again and prints them.
"""
from __future__ import annotations

import ctypes
import itertools
import math
import os
import random
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tiling_roofline_analysis_amd as tra
from tiling_roofline_analysis_amd import fused

TYPES = {"f32": 0, "bf16": 1, "f16": 2}

# M, N, K, type, layout, gated, padding, rows far apart
ROWS = [
    (1, 4, 4, "f32", "kn", 0, 0, 0), (70, 8288, 296, "f32", "kn", 0, 1, 0),
    (1550, 3964, 4, "f32", "kn", 0, 0, 0), (8251, 462, 130, "f32", "kn", 0, 0, 0),
    (10897, 8, 72, "f32", "kn", 0, 0, 0), (1, 2, 2, "f32", "kn", 0, 0, 1),
    (1, 72, 5552, "f32", "kn", 1, 0, 0), (1, 1368, 1312, "f32", "kn", 1, 0, 0),
    (1, 1889, 2074, "f32", "kn", 1, 0, 0), (1, 2056, 4776, "f32", "kn", 1, 0, 0),
    (1, 5128, 3824, "f32", "kn", 1, 0, 0), (1, 8996, 2082, "f32", "kn", 1, 1, 0),
    (1, 10976, 3000, "f32", "kn", 1, 0, 0), (17, 4, 4, "f32", "kn", 1, 0, 0),
    (27, 8731, 289, "f32", "kn", 1, 1, 0), (67, 2168, 2000, "f32", "kn", 1, 0, 0),
    (68, 1104, 12600, "f32", "kn", 1, 0, 0), (79, 6288, 2352, "f32", "kn", 1, 0, 0),
    (79, 15848, 528, "f32", "kn", 1, 0, 0), (381, 4, 8388, "f32", "kn", 1, 0, 0),
    (411, 2188, 4, "f32", "kn", 1, 0, 0), (433, 4135, 3, "f32", "kn", 1, 0, 0),
    (638, 68, 1424, "f32", "kn", 1, 0, 0), (1292, 1168, 4, "f32", "kn", 1, 0, 0),
    (1561, 2232, 72, "f32", "kn", 1, 0, 0), (1692, 1198, 133, "f32", "kn", 1, 0, 0),
    (1714, 1200, 208, "f32", "kn", 1, 0, 0), (1893, 6328, 72, "f32", "kn", 1, 0, 0),
    (2698, 40, 776, "f32", "kn", 1, 0, 0), (3153, 2600, 40, "f32", "kn", 1, 0, 0),
    (4121, 208, 2, "f32", "kn", 1, 0, 0), (5205, 4, 3150, "f32", "kn", 1, 0, 0),
    (19, 70, 3, "f32", "kn", 1, 0, 1), (20, 3, 167, "f32", "kn", 1, 0, 1),
    (1, 2, 2, "f32", "nk", 0, 0, 0), (1, 9544, 2704, "f32", "nk", 0, 0, 0),
    (34, 6256, 2672, "f32", "nk", 0, 0, 0), (65, 352, 8200, "f32", "nk", 0, 0, 0),
    (66, 4224, 7088, "f32", "nk", 0, 0, 0), (76, 1552, 4312, "f32", "nk", 0, 0, 0),
    (130, 5478, 708, "f32", "nk", 0, 0, 0), (231, 4, 4, "f32", "nk", 0, 0, 0),
    (737, 232, 5504, "f32", "nk", 0, 0, 0), (1690, 2432, 200, "f32", "nk", 0, 0, 0),
    (2761, 72, 720, "f32", "nk", 0, 0, 0), (3387, 1803, 4, "f32", "nk", 0, 0, 0),
    (8248, 456, 136, "f32", "nk", 0, 1, 0), (8615, 70, 331, "f32", "nk", 0, 0, 0),
    (9703, 328, 1168, "f32", "nk", 0, 0, 0), (9985, 66, 2, "f32", "nk", 0, 0, 0),
    (13937, 4, 84, "f32", "nk", 0, 0, 0), (1, 2, 2, "f32", "nk", 1, 0, 0),
    (1, 72, 12584, "f32", "nk", 1, 0, 0), (1, 1160, 2008, "f32", "nk", 1, 0, 0),
    (1, 1640, 4192, "f32", "nk", 1, 1, 0), (1, 1856, 1872, "f32", "nk", 1, 0, 0),
    (1, 1912, 6520, "f32", "nk", 1, 0, 0), (1, 3980, 2713, "f32", "nk", 1, 0, 0),
    (18, 104, 4, "f32", "nk", 1, 0, 0), (18, 8504, 368, "f32", "nk", 1, 0, 0),
    (18, 8751, 291, "f32", "nk", 1, 0, 0), (67, 3328, 3432, "f32", "nk", 1, 0, 0),
    (73, 2200, 2816, "f32", "nk", 1, 0, 0), (77, 15064, 584, "f32", "nk", 1, 0, 0),
    (290, 2, 8325, "f32", "nk", 1, 0, 0), (384, 4, 10804, "f32", "nk", 1, 0, 0),
    (588, 2437, 4, "f32", "nk", 1, 0, 0), (912, 1648, 2, "f32", "nk", 1, 0, 0),
    (1177, 1704, 216, "f32", "nk", 1, 0, 0), (1622, 1257, 161, "f32", "nk", 1, 1, 0),
    (1625, 1890, 4, "f32", "nk", 1, 0, 0), (2709, 40, 784, "f32", "nk", 1, 0, 0),
    (2967, 360, 72, "f32", "nk", 1, 0, 0), (6214, 8, 2592, "f32", "nk", 1, 0, 0),
    (9839, 608, 328, "f32", "nk", 1, 0, 0), (10083, 792, 40, "f32", "nk", 1, 0, 0),
    (20, 3, 171, "f32", "nk", 1, 1, 1), (20, 68, 3, "f32", "nk", 1, 0, 1),
    (164, 3, 2, "f32", "nk", 1, 0, 1), (66, 8232, 8, "bf16", "kn", 0, 0, 0),
    (199, 1368, 8664, "bf16", "kn", 0, 0, 0), (553, 7344, 520, "bf16", "kn", 0, 0, 0),
    (1813, 136, 5608, "bf16", "kn", 0, 0, 0), (1868, 2, 3210, "bf16", "kn", 0, 1, 0),
    (5457, 8, 2456, "bf16", "kn", 0, 0, 0), (5483, 456, 1432, "bf16", "kn", 0, 0, 0),
    (5736, 12064, 136, "bf16", "kn", 0, 0, 0), (7229, 3648, 136, "bf16", "kn", 0, 0, 0),
    (7954, 136, 8496, "bf16", "kn", 0, 0, 0), (13380, 8, 216, "bf16", "kn", 0, 0, 0),
    (1, 1288, 2984, "bf16", "kn", 1, 0, 0), (1, 1704, 1153, "bf16", "kn", 1, 1, 0),
    (1, 8744, 1712, "bf16", "kn", 1, 0, 0), (4, 14768, 72, "bf16", "kn", 1, 0, 0),
    (17, 8, 8, "bf16", "kn", 1, 0, 0), (18, 8200, 8, "bf16", "kn", 1, 0, 0),
    (65, 12384, 8, "bf16", "kn", 1, 0, 0), (67, 9432, 1712, "bf16", "kn", 1, 0, 0),
    (68, 1624, 8248, "bf16", "kn", 1, 0, 0), (69, 72, 7760, "bf16", "kn", 1, 0, 0),
    (137, 3256, 3664, "bf16", "kn", 1, 0, 0), (145, 2840, 3560, "bf16", "kn", 1, 0, 0),
    (158, 10944, 776, "bf16", "kn", 1, 1, 0), (198, 2752, 9584, "bf16", "kn", 1, 0, 0),
    (200, 4288, 1416, "bf16", "kn", 1, 0, 0), (201, 5016, 5424, "bf16", "kn", 1, 0, 0),
    (222, 3080, 2736, "bf16", "kn", 1, 0, 0), (257, 13520, 8, "bf16", "kn", 1, 0, 0),
    (261, 6552, 464, "bf16", "kn", 1, 0, 0), (339, 352, 11000, "bf16", "kn", 1, 1, 0),
    (758, 5480, 216, "bf16", "kn", 1, 1, 0), (905, 2703, 67, "bf16", "kn", 1, 0, 0),
    (1102, 3616, 416, "bf16", "kn", 1, 0, 0), (1256, 13104, 88, "bf16", "kn", 1, 0, 0),
    (1679, 216, 2408, "bf16", "kn", 1, 0, 0), (1826, 88, 4744, "bf16", "kn", 1, 0, 0),
    (2411, 67, 3357, "bf16", "kn", 1, 1, 0), (2803, 104, 6240, "bf16", "kn", 1, 0, 0),
    (2812, 1128, 72, "bf16", "kn", 1, 0, 0), (5937, 72, 15808, "bf16", "kn", 1, 0, 0),
    (8538, 1816, 2, "bf16", "kn", 1, 0, 0), (8989, 2, 1112, "bf16", "kn", 1, 1, 0),
    (10901, 72, 1456, "bf16", "kn", 1, 1, 0), (10916, 645, 140, "bf16", "kn", 1, 0, 0),
    (11923, 8, 2720, "bf16", "kn", 1, 0, 0), (15767, 24, 67, "bf16", "kn", 1, 0, 0),
    (1, 2, 2, "bf16", "nk", 0, 0, 0), (1, 8, 8, "bf16", "nk", 0, 0, 0),
    (65, 5216, 1007, "bf16", "nk", 0, 0, 0), (65, 8288, 8, "bf16", "nk", 0, 0, 0),
    (396, 608, 13136, "bf16", "nk", 0, 0, 0), (738, 4727, 864, "bf16", "nk", 0, 0, 0),
    (1153, 8, 8, "bf16", "nk", 0, 0, 0), (1666, 2, 2410, "bf16", "nk", 0, 0, 0),
    (2332, 2736, 72, "bf16", "nk", 0, 0, 0), (2333, 2, 2574, "bf16", "nk", 0, 0, 0),
    (3520, 72, 8224, "bf16", "nk", 0, 0, 0), (5463, 3192, 144, "bf16", "nk", 0, 0, 0),
    (6794, 2776, 200, "bf16", "nk", 0, 0, 0), (10903, 669, 346, "bf16", "nk", 0, 0, 0),
    (1, 2, 2, "bf16", "nk", 1, 0, 0), (1, 1296, 1160, "bf16", "nk", 1, 0, 0),
    (1, 2126, 1804, "bf16", "nk", 1, 0, 0), (1, 2459, 1178, "bf16", "nk", 1, 1, 0),
    (1, 4400, 4464, "bf16", "nk", 1, 0, 0), (17, 584, 8, "bf16", "nk", 1, 0, 0),
    (18, 8336, 8, "bf16", "nk", 1, 0, 0), (66, 8312, 1912, "bf16", "nk", 1, 0, 0),
    (68, 2762, 979, "bf16", "nk", 1, 0, 0), (75, 2504, 8328, "bf16", "nk", 1, 0, 0),
    (79, 12416, 8, "bf16", "nk", 1, 0, 0), (129, 11040, 560, "bf16", "nk", 1, 0, 0),
    (133, 5459, 1513, "bf16", "nk", 1, 0, 0), (137, 5832, 1584, "bf16", "nk", 1, 0, 0),
    (197, 8272, 8, "bf16", "nk", 1, 0, 0), (204, 4416, 5456, "bf16", "nk", 1, 0, 0),
    (325, 10967, 544, "bf16", "nk", 1, 0, 0), (385, 4728, 740, "bf16", "nk", 1, 0, 0),
    (844, 200, 9376, "bf16", "nk", 1, 0, 0), (1017, 34, 963, "bf16", "nk", 1, 0, 0),
    (1111, 1798, 2, "bf16", "nk", 1, 0, 0), (1139, 76, 7247, "bf16", "nk", 1, 0, 0),
    (1671, 2305, 265, "bf16", "nk", 1, 0, 0), (1711, 5544, 136, "bf16", "nk", 1, 1, 0),
    (2273, 7272, 104, "bf16", "nk", 1, 0, 0), (2686, 8, 4120, "bf16", "nk", 1, 0, 0),
    (2702, 104, 6024, "bf16", "nk", 1, 0, 0), (2764, 40, 2488, "bf16", "nk", 1, 0, 0),
    (2820, 104, 6600, "bf16", "nk", 1, 0, 0), (3550, 8, 9392, "bf16", "nk", 1, 0, 0),
    (4318, 6432, 144, "bf16", "nk", 1, 0, 0), (4340, 72, 14896, "bf16", "nk", 1, 0, 0),
    (5697, 104, 9736, "bf16", "nk", 1, 0, 0), (5784, 1135, 2, "bf16", "nk", 1, 0, 0),
    (6571, 816, 257, "bf16", "nk", 1, 0, 0), (8492, 40, 328, "bf16", "nk", 1, 0, 0),
    (9358, 200, 2904, "bf16", "nk", 1, 0, 0), (13243, 264, 8, "bf16", "nk", 1, 0, 0),
    (1, 2, 2, "f16", "kn", 0, 0, 0), (1, 8, 8, "f16", "kn", 0, 0, 0),
    (67, 3800, 8568, "f16", "kn", 0, 0, 0), (68, 905, 5460, "f16", "kn", 0, 0, 0),
    (130, 6816, 3680, "f16", "kn", 0, 0, 0), (220, 8936, 5501, "f16", "kn", 0, 0, 0),
    (449, 2704, 8880, "f16", "kn", 0, 0, 0), (503, 776, 9456, "f16", "kn", 0, 0, 0),
    (957, 5796, 67, "f16", "kn", 0, 0, 0), (1153, 8, 8, "f16", "kn", 0, 0, 0),
    (1612, 2, 2559, "f16", "kn", 0, 0, 0), (1677, 710, 2376, "f16", "kn", 0, 0, 0),
    (2179, 8, 1360, "f16", "kn", 0, 0, 0), (3659, 8, 1040, "f16", "kn", 0, 0, 0),
    (8814, 3632, 3, "f16", "kn", 0, 0, 0), (10962, 136, 8296, "f16", "kn", 0, 0, 0),
    (11977, 8, 240, "f16", "kn", 0, 0, 0), (1, 904, 1616, "f16", "kn", 1, 0, 0),
    (1, 1682, 1671, "f16", "kn", 1, 0, 0), (1, 8296, 1880, "f16", "kn", 1, 0, 0),
    (1, 9712, 240, "f16", "kn", 1, 0, 0), (17, 2, 321, "f16", "kn", 1, 0, 0),
    (17, 8200, 8, "f16", "kn", 1, 0, 0), (68, 4120, 5480, "f16", "kn", 1, 0, 0),
    (130, 8208, 8, "f16", "kn", 1, 0, 0), (136, 10920, 488, "f16", "kn", 1, 0, 0),
    (151, 737, 10889, "f16", "kn", 1, 0, 0), (160, 5463, 1518, "f16", "kn", 1, 0, 0),
    (164, 2728, 3480, "f16", "kn", 1, 0, 0), (195, 3120, 2816, "f16", "kn", 1, 0, 0),
    (259, 5464, 675, "f16", "kn", 1, 0, 0), (325, 2896, 1408, "f16", "kn", 1, 0, 0),
    (451, 648, 4448, "f16", "kn", 1, 0, 0), (514, 7272, 8, "f16", "kn", 1, 0, 0),
    (706, 136, 8312, "f16", "kn", 1, 0, 0), (725, 5448, 328, "f16", "kn", 1, 1, 0),
    (789, 8233, 3, "f16", "kn", 1, 0, 0), (1456, 5480, 136, "f16", "kn", 1, 0, 0),
    (1574, 1287, 2, "f16", "kn", 1, 0, 0), (1674, 278, 69, "f16", "kn", 1, 0, 0),
    (1900, 72, 5080, "f16", "kn", 1, 0, 0), (2702, 1176, 72, "f16", "kn", 1, 0, 0),
    (3337, 112, 2376, "f16", "kn", 1, 1, 0), (3601, 560, 648, "f16", "kn", 1, 1, 0),
    (4274, 72, 13856, "f16", "kn", 1, 0, 0), (4384, 7152, 152, "f16", "kn", 1, 0, 0),
    (4692, 232, 840, "f16", "kn", 1, 0, 0), (5534, 112, 9120, "f16", "kn", 1, 0, 0),
    (6901, 8, 4792, "f16", "kn", 1, 0, 0), (9365, 2, 1074, "f16", "kn", 1, 0, 0),
    (9414, 448, 560, "f16", "kn", 1, 0, 0), (15846, 8, 72, "f16", "kn", 1, 0, 0),
    (1, 2, 8, "f16", "kn", 1, 0, 1), (129, 8, 5448, "f16", "nk", 0, 0, 0),
    (516, 686, 7235, "f16", "nk", 0, 0, 0), (1103, 7200, 392, "f16", "nk", 0, 0, 0),
    (6000, 8, 1288, "f16", "nk", 0, 0, 0), (6584, 1685, 260, "f16", "nk", 0, 0, 0),
    (8588, 208, 5416, "f16", "nk", 0, 0, 0), (1, 2, 2, "f16", "nk", 1, 0, 0),
    (1, 1687, 1173, "f16", "nk", 1, 0, 0), (1, 4496, 4312, "f16", "nk", 1, 0, 0),
    (1, 8288, 2120, "f16", "nk", 1, 1, 0), (2, 72, 15056, "f16", "nk", 1, 0, 0),
    (17, 8232, 8, "f16", "nk", 1, 0, 0), (18, 584, 8, "f16", "nk", 1, 0, 0),
    (67, 2584, 8208, "f16", "nk", 1, 0, 0), (67, 4344, 4200, "f16", "nk", 1, 0, 0),
    (68, 2796, 1001, "f16", "nk", 1, 0, 0), (68, 9360, 1760, "f16", "nk", 1, 0, 0),
    (69, 12488, 8, "f16", "nk", 1, 0, 0), (129, 11128, 688, "f16", "nk", 1, 0, 0),
    (132, 1736, 5624, "f16", "nk", 1, 0, 0), (168, 5448, 1680, "f16", "nk", 1, 1, 0),
    (196, 1464, 6400, "f16", "nk", 1, 0, 0), (274, 1152, 6040, "f16", "nk", 1, 0, 0),
    (513, 224, 7288, "f16", "nk", 1, 0, 0), (585, 3327, 779, "f16", "nk", 1, 0, 0),
    (1089, 74, 7267, "f16", "nk", 1, 0, 0), (1096, 3648, 488, "f16", "nk", 1, 0, 0),
    (1422, 10968, 80, "f16", "nk", 1, 0, 0), (1643, 5448, 143, "f16", "nk", 1, 0, 0),
    (1804, 2312, 136, "f16", "nk", 1, 0, 0), (2214, 1355, 2, "f16", "nk", 1, 0, 0),
    (2832, 40, 2504, "f16", "nk", 1, 0, 0), (4329, 67, 13328, "f16", "nk", 1, 0, 0),
    (5470, 104, 10976, "f16", "nk", 1, 0, 0), (5474, 1680, 8, "f16", "nk", 1, 0, 0),
    (5486, 760, 248, "f16", "nk", 1, 1, 0), (6172, 1392, 208, "f16", "nk", 1, 0, 0),
    (6796, 144, 1800, "f16", "nk", 1, 0, 0), (6839, 8, 4808, "f16", "nk", 1, 0, 0),
    (8521, 40, 336, "f16", "nk", 1, 0, 0), (8568, 672, 208, "f16", "nk", 1, 0, 0),
    (9080, 532, 2, "f16", "nk", 1, 1, 0), (13085, 152, 640, "f16", "nk", 1, 0, 0),
]


def pitch(cols, row):
    """Elements from one row of a matrix to the next."""
    *_, dtype, _, _, pad, far = row
    return (1 << 22) // (4 if dtype == "f32" else 2) + 1 if far else cols + pad


def packed(row, p=None):
    """The packed arguments of a row's forward and backward call; p: addresses by
    name, or none that are read."""
    M, N, K, dtype, layout, gated, _, _ = row
    nk = int(layout == "nk")
    at = dict(X=1 << 45, W=1 << 50, W2=1 << 51, Y=1 << 52, dY=1 << 44, Z=1 << 46, dX=1 << 53,
              dW=1 << 54, dW2=1 << 55) if p is None else p
    ldw, W2, width = pitch(K if nk else N, row), at["W2"] if gated else 0, N * (1 + gated)
    fwd = fused._ARGS.pack(TYPES[dtype], 1, nk, gated, M, N, K, at["X"], pitch(K, row), at["W"],
                           W2, ldw, 0, 0, 0, at["Y"], N, 0, 0, 0, 0)
    bwd = fused._GRAD_ARGS.pack(TYPES[dtype], 1 if gated else 0, nk, gated, M, N, K, at["dY"],
                                pitch(N, row), at["Z"], width, at["X"], pitch(K, row), at["W"], W2,
                                ldw, at["dX"], K, at["dW"], at["dW2"] if gated else 0,
                                K if nk else N, 0, 0, 0)
    return fwd, bwd


def described(packed_args, name):
    buf = ctypes.create_string_buffer(512)
    assert getattr(tra.load(), name)(packed_args, buf, 512) == tra.TRA_OK
    return dict(kv.split("=") for kv in buf.value.decode().split())


def plans(row, p=None):
    """What a row launches: (type, form, gated, kernel, tile, stages, bytes of direct
    loads, how split) of the forward product, dX and dW."""
    _, _, _, dtype, layout, gated, _, _ = row
    fwd, bwd = packed(row, p)
    f = described(fwd, "tra_linear_describe")
    b = described(bwd, "tra_linear_backward_describe")

    def key(d, prefix, form, gated):
        d = {k[len(prefix):]: v for k, v in d.items() if k.startswith(prefix)}
        if d["kernel"] == "linear_few" or d["splits"] == "1":
            split = "no"
        else:
            split = "all" if d["whole"] == "0" else "last"
        return (dtype, form, gated, d["kernel"], d["tile"], int(d["stages"]), int(d["load_bytes"]),
                split)

    nk = layout == "nk"
    return [key(f, "", "KK" if nk else "KN", gated), key(b, "dx_", "KN" if nk else "KK", 0),
            key(b, "dw_", "NN", 0)]


def instances():
    """Every kernel instance: the keys of plans() without the split.  Forms: KK, both
    operands k-contiguous; KN, the second not; NN, neither."""
    for dtype, (form, gated) in itertools.product(
            TYPES, (("KK", 0), ("KK", 1), ("KN", 0), ("KN", 1), ("NN", 0))):
        tile = (dtype, form, gated, "linear_tile")
        for size, stages in (("128x128", (2, 4)), ("64x128", (3, 6)), ("64x64", (3, 6))):
            for s in stages:
                yield (*tile, size, s, 16)
        if dtype == "f32":
            yield from ((*tile, "64x64", 2, 0), (*tile, "64x128", 3, 4), (*tile, "64x64", 3, 4))
        else:
            for size in ("128x128", "64x128", "64x64"):
                yield (*tile, size, 2, 0)
            yield (*tile, "256x256", 2, 16)
        if form != "NN":
            cols = 16 if form == "KK" else 64 // (4 if dtype == "f32" else 2)
            yield (dtype, form, gated, "linear_few", f"16x{cols * (1 + gated)}", 0, 0)


# (instance, split) pairs that the search finds calls for
PAIRS = 395


def search(seconds):
    """The cheapest random call for every (instance, split) found in a while, and of
    those calls a few that cover all."""
    import time
    rng, best, end = random.Random(1), {}, time.time() + seconds

    def size(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi))))

    def cost(row):
        return 2.0 * row[0] * row[1] * row[2] * (1 + row[5]) + 1e3 * sum(row[:3])

    while time.time() < end:
        hi = rng.choice((400, 2000, 6000, 9000, 16000))
        M, N, K = size(1, hi), size(2, hi), size(2, hi)
        if 2.0 * M * N * K > 8e11 or max(M * N, N * K, M * K) > 1.4e8:
            continue
        if rng.random() < 0.7:
            N, K = -(-N // 8) * 8, -(-K // 8) * 8
        far = int(max(M, N, K) < 300 and rng.random() < 0.06)
        row = (M, N, K, rng.choice(list(TYPES)), rng.choice(("kn", "nk")), rng.choice((0, 1)),
               int(rng.random() < 0.17), far)
        for k in plans(row):
            if k not in best or cost(row) < cost(best[k]):
                best[k] = row
    covers = {row: set(plans(row)) for row in best.values()}
    left, rows = set(best), []
    while left:
        row = max(covers, key=lambda r: (len(covers[r] & left) / (1 + cost(r) / 3e9), -cost(r)))
        rows.append(row)
        left -= covers[row]
    return sorted(rows, key=lambda r: (TYPES[r[3]], *r[4:])), len(best)


if __name__ == "__main__":
    found, pairs = search(float(sys.argv[1]) if len(sys.argv) > 1 else 300.0)
    for row in found:
        print(f"    {row},")
    print(f"PAIRS = {pairs}")
