"""Rows, columns and entries of products in 4 bits whose rows end with a group of scales of a single period (1024 n + 256
stored entries, n from 2 on), on large tiles in one go (test_mx_loads.py holds them to that)."""
CUT = [(4096, 4096, 2304), (4100, 4093, 3300), (4096, 4096, 5376), (2048, 5000, 4200)]

# One kind of kernel each: few rows, whole and split, 128-row tiles, whole and split (gated: large ones), large ones, whole and split.
FEW, FEW_SPLIT, TILE, TILE_SPLIT, LARGE, LARGE_SPLIT = PLACES = [
    (40, 200, 900), (162, 139, 23916), (1500, 700, 2100), (150, 2745, 21624), (2500, 4100, 2100), (1438, 1387, 22308)]
