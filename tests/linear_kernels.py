"""Products of sv_linear by the kernel that they take, one shape or more for
each: odd sizes that end inside tiles and rounds.  tests/test_linear_pick.py
holds the choice to this table, so that a change of the rule cannot leave a
kernel untested."""

ROWS_16, ROWS_32 = -1, -2  # up to 16 rows, 16 and 32 columns a workgroup; from 0 on, the tiles

# kernel, M, N, K
KERNELS = [
    (ROWS_32, 5, 8315, 320),
    (ROWS_16, 7, 1005, 704),
    (0, 45, 165, 1088),      # 32 x 32
    (1, 74, 3093, 320),      # 32 x 64
    (2, 137, 3531, 320),     # 64 x 64
    (3, 28, 16887, 320),     # 64 x 128
    (3, 9, 26877, 4160),     # and with few rows that are long
    (4, 145, 11011, 320),    # 128 x 128
    (5, 31, 37101, 320),     # 128 x 256
    (6, 185, 34923, 320),    # 192 x 256
    (7, 408, 22467, 320),    # 224 x 256
]
