"""Calls of fp8_linear and fp4_moe_experts by the kernel that they reach on 256 CUs. tests/test_routes_cpu.py checks that they do
(choices.hpp decides), tests/test_gpu_routes.py checks their results."""

# shapes of choices.hpp, by their place there
SPLIT16, SPLIT16X32, SPLIT32, RING64, RING128X64, RING128, RING128_TWO, TURNS256 = range(8)

# fp8_linear (M, N, K): K of enough blocks that the ring's buffers are used again, an odd number of them and past 64 of them (W's
# scales are loaded 64 at a time); M and N end inside a tile, N odd
LINEAR = {
    RING64: [(61, 14333, 1152), (63, 13001, 896), (50, 16001, 1280), (64, 14001, 8320)],
    RING128X64: [(120, 14333, 1152), (127, 14001, 640), (100, 13999, 8448), (129, 8001, 8320)],
    RING128: [(190, 16001, 1152), (230, 14333, 640), (200, 14001, 8320)],
    RING128_TWO: [(300, 14333, 1152), (350, 13001, 640), (300, 14001, 8320)],
    TURNS256: [(1000, 14333, 1152), (770, 13003, 640), (1030, 12301, 8320)],
}
# fp8_linear of few blocks of K, M and N ragged: one of every shape, for what must not leave its rows or Y
EDGES = {
    SPLIT16: (7, 4101, 640), SPLIT16X32: (37, 4099, 640), SPLIT32: (60, 4001, 640), RING64: (61, 14333, 640),
    RING128X64: (127, 14001, 640), RING128: (230, 14333, 640), RING128_TWO: (350, 13001, 640), TURNS256: (770, 13003, 640),
}

# fp4_moe_experts T, k, E, D, I, block, waves of a workgroup (up, down), and the tokens of the used experts: 1 to 4 fragments of 4
# tokens in a pass, and up to three passes. Rows of scales longer than 4096 elements take several windows of LDS.
EXPERTS = [
    (40, 2, 64, 4224, 512, 32, 2, 1, (21, 16, 11, 7, 4, 1)),   # two windows, the last one starting at scale byte 4
    (40, 2, 64, 7168, 512, 128, 2, 1, (12, 1, 6, 18, 2)),      # two windows, the last one at 96
    (45, 2, 64, 8320, 512, 16, 2, 1, (15, 33, 3, 9)),          # three windows; three passes
    (45, 2, 64, 1024, 4352, 64, 1, 2, (35, 2, 16, 5, 9)),      # two windows in the second product
    (64, 2, 32, 2048, 1664, 32, 2, 2, (21, 13, 8, 4, 16, 30)),
    (64, 2, 64, 1024, 512, 64, 1, 1, (21, 13, 8, 4, 16, 30)),
    (40, 2, 8, 4224, 256, 32, 8, 8, (21, 16, 11, 7, 4, 1)),
    (50, 2, 6, 640, 4224, 128, 8, 8, (33, 16, 11, 7, 4, 1)),
]
