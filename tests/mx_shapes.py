"""Rows, columns and entries of products that reach every compiled kernel of the microscaled products,
whole and, where any sizes lead to it, with a split contraction (test_mx_plans.py holds them to that)."""
SHAPES = [(1, 4445, 3106), (2, 17, 32), (3, 17, 15671), (3, 1449, 20369), (36, 543, 30522), (84, 325, 25329), (145, 137, 30203),
          (168, 803, 3715), (198, 49, 29314), (234, 1025, 32), (255, 793, 33), (325, 247, 28323), (447, 35, 28568),
          (1257, 19, 32438), (1438, 1387, 22308), (1629, 43, 28294), (1899, 3273, 264), (2053, 101, 24935), (2234, 33, 1042),
          (2693, 1413, 8960), (2874, 265, 32), (3268, 139, 292), (3447, 3637, 276), (3845, 389, 33), (4200, 35, 5595),
          (4446, 41, 333), (4720, 33, 34)]
# Ends of the rows, of a group of scales (512 and 1024 entries), of tiles and of a round of the XCDs.
EDGES = [(256, 256, 256), (257, 257, 512), (511, 513, 768), (512, 264, 1024), (2049, 2060, 1280), (1030, 4100, 1536), (2304, 2297, 2049)]
