"""Sizes (tokens, K, N) of the product tests, by the form of the kernel that
they are for; test_mx_geometry checks on the CPU that they take it."""

# CTA pairs, whatever the type of x; the tokens split into tiles of
PAIRS = [
    (60, 1000, 7100),      # 64
    (128, 2560, 7000),     # 64, two of them
    (190, 256, 19000),     # 192
    (110, 640, 19000),     # 128
    (150, 384, 10000),     # 160
    (200, 128, 10100),     # 224
    (300, 1000, 5000),     # 160, from an offset of 32 on
    (384, 1500, 9000),     # 192
    (380, 256, 4999),      # 192
    (420, 2048, 4900),     # 224, over three scale tiles
    (700, 640, 3400),      # 256
    (1200, 300, 2050),     # 256, two rows in the last row tile
    (2500, 640, 4200),     # 256, three tiles to a pair
    (150, 256, 50000),     # 160, three tiles to a pair
    (420, 4224, 16001),    # 224, two tiles to a pair, an odd number of scale tiles
    # Up to 128, two blocks of K a stage:
    (192, 4224, 9000),     # 96, two of them; an odd number of blocks, the last one half of 4-bit x
    (300, 1152, 4100),     # 96, from offsets of 96, 64 and 32 in a scale tile on
    (380, 4096, 2100),     # 64, six of them
    (600, 1664, 2500),     # 128, five of them
    (128, 128, 7000),      # 64, less than a block
    (128, 640, 40000),     # 128, three tiles to a pair, an odd number of blocks
    (100, 384, 50000),     # 128, three tiles to a pair
]

# Single CTAs, K split by (the splits with 4-bit and with 8-bit x)
SPLIT = [
    (1, 32, 5),            # 1, 1
    (1, 4096, 300),        # 8, 8
    (3, 4224, 257),        # 6, 7
    (16, 2560, 130),       # 5, 7
    (17, 4096, 11008),     # 3, 3
    (20, 2560, 7000),      # 4, 4
    (24, 8192, 8000),      # 4, 4
    (20, 300, 20000),      # 1, 1
    (64, 8192, 1200),      # 8, 8
    (200, 8192, 300),      # 8, 8: two tiles of tokens
    (513, 11008, 129),     # 4, 8: five, the last of one token
]

ANY = [
    (128, 4096, 600), (256, 4224, 520),
    (1, 1, 1), (1, 128, 128), (2, 100, 129), (7, 1000, 31), (8, 640, 384), (9, 256, 1000), (17, 384, 256),
    (31, 1056, 77), (32, 512, 640), (33, 640, 5000), (33, 896, 300), (64, 1024, 128), (65, 300, 200), (90, 2560, 7000),
    (96, 256, 130), (100, 2560, 140), (127, 130, 250), (128, 512, 256), (129, 512, 300), (160, 1408, 270),
    (200, 384, 520), (255, 260, 129), (256, 1024, 128), (257, 128, 385), (300, 777, 333), (385, 640, 513),
    (513, 1152, 260), (1030, 256, 700)]
