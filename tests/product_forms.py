"""Sizes at which each form of the tensor-core product runs (csrc/product_tc.cuh, TcConfig), with
ragged edges: the GPU tests run them, and a CPU test sees that each form is reached."""

PAIR256, SINGLE128, SINGLE64, SWAP64, SWAP32, SWAP16, PAIR128 = range(7)
TILE = {PAIR256: (256, 256, 76), SINGLE128: (128, 128, 152), SINGLE64: (128, 64, 152), SWAP64: (64, 128, 152),
        SWAP32: (32, 128, 304), SWAP16: (16, 128, 304), PAIR128: (256, 128, 76)}      # rows, columns, at one time

# m, n, k, dtype_in, dtype_out, form
FORMS = [
    (1300, 2104, 704, "bf16", "bf16", PAIR256), (2600, 4200, 712, "bf16", "bf16", PAIR256),
    (1300, 2104, 704, "bf16", "f32", PAIR256), (2600, 4200, 712, "bf16", "f32", PAIR256),
    (4100, 4104, 16, "bf16", "bf16", PAIR256), (4100, 4090, 16, "bf16", "f32", PAIR256),
    (700, 2056, 1032, "bf16", "bf16", PAIR128), (700, 2056, 1032, "bf16", "f32", PAIR128),
    (2600, 4200, 200, "f32", "f32", PAIR128), (2600, 4200, 200, "f32", "bf16", PAIR128),
    (1030, 4100, 264, "bf16", "bf16", SINGLE128), (1030, 4100, 264, "bf16", "f32", SINGLE128),
    (1030, 4100, 264, "f32", "f32", SINGLE128), (1030, 4100, 264, "f32", "bf16", SINGLE128),
    (600, 1000, 300, "bf16", "bf16", SINGLE64), (600, 1000, 300, "bf16", "f32", SINGLE64),
    (300, 300, 300, "f32", "f32", SINGLE64), (300, 300, 300, "f32", "bf16", SINGLE64),
    (64, 32000, 520, "bf16", "bf16", SWAP64), (50, 32010, 520, "bf16", "f32", SWAP64),
    (50, 32010, 520, "f32", "f32", SWAP64), (50, 8000, 520, "f32", "bf16", SWAP64),
    (32, 64000, 136, "bf16", "bf16", SWAP32), (27, 64010, 136, "bf16", "f32", SWAP32),
    (27, 32010, 136, "f32", "f32", SWAP32), (16, 64000, 136, "bf16", "bf16", SWAP16),
    (13, 64010, 136, "bf16", "f32", SWAP16),
]


def tiles(m, n, form):
    rows, cols, _ = TILE[form]
    return -(-m // rows) * (-(-n // cols))
