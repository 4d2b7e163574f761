"""Sizes of the fused and grouped products that take each of their kernels, named by the kernel's workgroup tile (rows of S,
tokens): tests run on every one of them, and a test without a GPU asserts that they still do take it."""
import torch

F32, BF16 = torch.float32, torch.bfloat16

# type, experts (None: one layer), tile, M, n_in, n_out, r
SIZES = [
    (BF16, None, (16, 16), 13, 1056, 203, 48), (BF16, None, (32, 16), 15, 96, 8200, 16), (BF16, None, (16, 32), 100, 96, 1003, 80),
    (BF16, None, (32, 32), 100, 2080, 2050, 48), (BF16, None, (128, 64), 250, 2080, 4090, 80), (BF16, None, (128, 64), 256, 4096, 4096, 64),
    (BF16, None, (256, 128), 2000, 1056, 4096, 80), (BF16, None, (256, 128), 1900, 1024, 4098, 144),
    (BF16, None, (512, 128), 4000, 992, 2050, 48), (BF16, None, (512, 128), 4000, 1024, 4096, 144),
    (BF16, 4, (16, 16), 13, 1056, 40, 48), (BF16, 4, (32, 16), 60, 96, 4100, 16), (BF16, 4, (16, 32), 500, 96, 200, 80),
    (BF16, 4, (32, 32), 300, 2080, 1032, 48), (BF16, 4, (128, 64), 700, 1056, 1003, 80), (BF16, 4, (256, 128), 4000, 1056, 2048, 144),
    (BF16, 4, (512, 128), 700, 992, 8200, 80), (BF16, 4, (512, 128), 690, 1024, 8197, 144),
    (F32, None, (16, 16), 13, 1056, 203, 48), (F32, None, (16, 32), 200, 1056, 1003, 80), (F32, None, (128, 64), 700, 1056, 1003, 80),
    (F32, 4, (16, 16), 13, 1056, 40, 48), (F32, 4, (16, 32), 300, 1056, 520, 80), (F32, 4, (128, 64), 700, 1056, 1003, 144),
]
IDS = ["-".join(map(str, (str(d)[6:], e, "%dx%d" % t, M, k, n, r))) for d, e, t, M, k, n, r in SIZES]
