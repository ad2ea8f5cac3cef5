"""Calls that take every form of the heads' kernel and of the attention's.  The host test works out, with the library's own
rules, which form each of them takes, and that none is left out; the GPU tests run them."""

KINDS = ["bf16", "int8", "fp8"]

# Rotations alone (unrounded): T, heads, dim, dims, interleaved, norm, as in test_heads_gpu.py.
ROPE = [
    (1025, 2, 256, 256, False, False), (1025, 1, 256, 96, True, True), (1027, 1, 144, 144, False, True),     # heads of 32 lanes, 4 tokens
    (8200, 1, 128, 128, False, True), (8200, 1, 80, 48, True, False), (8197, 1, 128, 64, True, True),        # of 16 lanes, 16 tokens
    (1030, 4, 128, 128, True, False), (1030, 3, 96, 96, False, True),                                        # of 16 lanes, 4 tokens
    (8200, 2, 64, 64, False, True), (8193, 1, 64, 32, True, False), (1030, 8, 64, 64, False, False),         # of 8 lanes
    (1029, 5, 48, 32, True, True), (3, 9, 64, 64, True, False), (1030, 9, 64, 64, False, True),
    (2, 5, 128, 128, True, True), (2, 3, 256, 256, False, False), (1030, 3, 256, 128, True, False),
]

# Writes: T, heads, kv_heads, dim, page, dims (0: no rotation), interleaved, norm; each with every kind.
WRITE = [
    (1030, 0, 1, 256, 32, 256, False, True), (1030, 0, 1, 256, 32, 128, True, False), (1027, 0, 1, 144, 16, 0, False, True),   # 32 lanes, 4 tokens
    (1030, 2, 1, 128, 48, 128, False, True), (1031, 0, 2, 80, 16, 48, True, False), (1030, 0, 2, 128, 64, 0, False, False),    # 16 lanes, 4 tokens
    (8200, 0, 1, 64, 48, 64, False, False), (8200, 0, 1, 64, 16, 32, True, True), (8195, 0, 1, 48, 32, 0, False, True),        # 8 lanes, 16 tokens
    (1030, 4, 2, 64, 32, 64, False, True), (1030, 1, 1, 64, 16, 64, True, False), (1033, 0, 4, 32, 16, 0, False, False),       # 8 lanes, 4 tokens
    (5, 8, 2, 256, 16, 256, False, True), (5, 2, 2, 256, 16, 64, True, False), (5, 0, 2, 256, 16, 0, False, False),
    (7, 8, 2, 128, 16, 128, False, True), (7, 8, 2, 128, 16, 128, True, False), (7, 0, 2, 128, 16, 0, False, False),
    (6, 9, 3, 64, 16, 64, False, True), (6, 9, 3, 64, 16, 64, True, False), (6, 0, 3, 64, 16, 0, False, False),
    (1030, 5, 1, 128, 16, 128, False, False), (1030, 7, 1, 64, 16, 64, True, True),     # a head too many for several tokens
]

SHORT = [0, 1, 33, 255, 256, -1, 16, 64, 130]
MEDIUM = [i * 389 % 1024 + 1 for i in range(30)] + [0, -1, 1024, 1008]

# Attention: lengths, heads, kv_heads, dim, page, columns, window; each with every kind.
ATTENTION = [
    # one launch: a table of at most 256 tokens (512 up to 64 channels)
    (SHORT, 4, 2, 16, 16, 16, 0), (SHORT, 17, 1, 64, 64, 4, 50), (SHORT, 8, 2, 80, 16, 16, 0), (SHORT, 17, 1, 128, 16, 16, 0),
    (SHORT, 32, 8, 128, 32, 8, 100), (SHORT, 40, 1, 112, 64, 4, 0), (SHORT, 4, 2, 144, 16, 16, 0), (SHORT, 34, 2, 256, 16, 16, 0),
    (SHORT, 8, 8, 256, 128, 2, 70), (SHORT, 3, 1, 192, 48, 5, 0),
    # one launch: up to 2048 tokens where the sequences and groups of heads are 128 and more
    (MEDIUM, 4, 4, 64, 16, 64, 0), (MEDIUM, 8, 4, 128, 16, 64, 0), (MEDIUM, 4, 4, 80, 32, 64, 300), (MEDIUM, 4, 4, 256, 64, 16, 0),
    # items of several workgroups, joined
    (SHORT, 4, 2, 64, 16, 40, 0), (SHORT, 17, 1, 128, 16, 17, 100), (SHORT, 8, 2, 256, 16, 17, 0), ([1024, 0, 700, -1, 33], 8, 2, 128, 16, 64, 0),
    ([1024, 0, 700, -1, 33], 6, 2, 192, 16, 64, 500), ([2048, 3], 4, 2, 48, 16, 128, 0),
]
