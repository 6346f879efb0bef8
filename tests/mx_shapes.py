"""Rows, columns and entries of products that reach every compiled kernel of the microscaled products,
whole and, where any sizes lead to it, with a split contraction (test_mx_plans.py holds them to that)."""
SHAPES = [(1, 17, 21292), (1, 1403, 31555), (2, 17, 32), (3, 1449, 20369), (56, 2139, 35), (112, 2311, 74), (150, 2745, 21624),
          (153, 437, 33), (162, 139, 23916), (216, 65, 21747), (234, 1025, 32), (1438, 1387, 22308), (1535, 17, 36179),
          (2092, 43, 15998), (2448, 17, 23515), (2805, 659, 15989), (2874, 265, 32), (3268, 139, 292), (3447, 3637, 276),
          (3845, 389, 33), (4106, 73, 2089), (4124, 35, 536), (4218, 77, 39), (4446, 41, 333)]
# Ends of the rows, of a group of scales (512 and 1024 entries), of tiles and of a round of the XCDs.
EDGES = [(256, 256, 256), (257, 257, 512), (511, 513, 768), (512, 264, 1024), (2049, 2060, 1280), (1030, 4100, 1536), (2304, 2297, 2049)]
