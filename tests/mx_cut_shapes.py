"""Rows, columns and entries of products in 4 bits whose rows end with a group of scales of a single period (1024 n + 256
stored entries, n from 2 on), on large tiles in one go (test_mx_loads.py holds them to that)."""
CUT = [(4096, 4096, 2304), (4100, 4093, 3300), (4096, 4096, 5376), (2048, 5000, 4200)]
