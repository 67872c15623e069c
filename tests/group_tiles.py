"""Sizes that reach every instance of the grouped rows' products, and what the library
says that a call takes (256 CUs).  The choices are fitted to times and may move:
test_group_tiles.py fails when a size no longer reaches its instance."""
import ctypes

import dense_gemm_linear_amd as dg

FORWARD, DX, DW, ADAPTERS = range(4)


def choice(op, T, k, groups, N, K, R=0):
    text = ctypes.create_string_buffer(64)
    i64 = ctypes.c_int64
    dg.lib.dg_group_choice(ctypes.c_int(op), i64(T), i64(k), i64(groups), i64(N), i64(K), i64(R), ctypes.c_int(256),
                           text, ctypes.c_size_t(64))
    return text.value.decode()


# tile, T, k, groups, N, K: N odd and N a multiple of 8 (stores and multipliers by the
# piece), K with a partly filled last k-tile (but 256x128: no such K takes it)
FORWARDS = [("16x32", 3, 1, 3, 133, 1032), ("16x32", 3, 1, 3, 136, 568),
            ("32x64", 2, 3, 6, 5787, 528), ("32x64", 3, 3, 6, 5784, 528),
            ("64x64", 341, 3, 49, 517, 560), ("64x64", 341, 3, 49, 520, 568),
            ("64x128", 85, 4, 21, 2641, 520), ("64x128", 85, 4, 21, 2640, 520),
            ("128x64", 5849, 3, 23, 9, 536), ("128x64", 5849, 3, 23, 56, 536),
            ("128x128", 721, 2, 42, 1351, 552), ("128x128", 721, 2, 42, 1352, 544),
            ("128x128 deep", 92, 4, 17, 1491, 552), ("128x128 deep", 92, 4, 17, 1488, 520),
            ("256x128", 4941, 1, 47, 451, 544), ("256x128", 4941, 1, 47, 456, 544),
            ("256x256", 2472, 3, 34, 1155, 296), ("256x256", 904, 2, 20, 2688, 608)]
# dX sums over N and has K columns
DXS = [("32x128", 20, 1, 3, 1032, 200), ("64x128", 1145, 1, 50, 496, 408), ("128x128 transposed", 1609, 1, 30, 144, 432),
       ("256x128", 2604, 2, 54, 776, 392), ("256x256", 2096, 2, 55, 648, 968)]
DWS = [("128x128 transposed", 60, 2, 6, 136, 200), ("256x128", 1511, 1, 1, 264, 392)]
# T, groups, N, K, R
ADAPTER_SIZES = [("token 1", 1, 4, 1001, 264, 32), ("token 2", 1, 4, 4313, 264, 40), ("token 3", 1, 8, 8483, 272, 112),
                 ("token 4", 1, 7, 100839, 272, 72), ("token 4", 1, 3, 14337, 520, 16),
                 ("slices 32", 130, 6, 5765, 936, 24), ("slices 64", 33, 5, 600, 4104, 24),
                 ("slices 128", 529, 9, 4241, 584, 8), ("slices 128", 67, 49, 8764, 584, 32),
                 ("slices 128", 66, 42, 8310, 648, 112),
                 # up to 64 rows a tile and 32 ranks: of many adapters summed row by row, of few
                 # as steps of the matrix cores
                 ("whole 16x32, inner 32x16", 2438, 512, 9, 272, 24), ("whole 32x64, inner row", 32, 32, 28673, 2056, 16),
                 ("whole 64x64, inner 32x16", 2188, 512, 237, 872, 24),
                 ("whole 64x128, inner row", 38, 96, 160811, 288, 24),
                 ("whole 16x32, inner 32x16", 2438, 58, 9, 272, 24), ("whole 32x64, inner row", 2, 6, 141613, 368, 24),
                 ("whole 64x64, inner 32x16", 2189, 35, 237, 872, 24),
                 ("whole 64x128, inner row", 37, 37, 160811, 288, 24),
                 # more ranks
                 ("whole 16x32, inner 32x16", 294, 4, 9, 552, 208), ("whole 32x64, inner 32x32", 620, 39, 193, 536, 224),
                 ("whole 64x64, inner 64x64", 3420, 17, 133, 296, 248),
                 ("whole 64x128, inner 32x16", 171, 23, 8808, 296, 256), ("whole 128x64, inner 32x32", 3376, 8, 129, 272, 40),
                 ("whole 128x128, inner 32x64", 4758, 13, 793, 264, 64),
                 ("whole 128x128 deep, inner 16x16", 264, 12, 5579, 264, 56),
                 ("whole 256x128, inner 32x32", 453, 53, 9232, 2504, 240),
                 ("whole 256x256, inner 16x16", 962, 7, 8313, 272, 16),
                 ("whole 256x256, inner 64x64", 2708, 8, 3049, 264, 256),
                 ("whole 128x64, inner 64x16", 4313, 17, 105, 264, 40), ("whole 128x128 deep, inner 64x32", 4102, 3, 545, 264, 80)]
