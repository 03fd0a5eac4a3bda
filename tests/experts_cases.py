"""A problem for every form of the products by group and of block-scaled 8-bit floats, named
by the library's plan queries: the host tests hold the plan to them, the GPU tests run them."""
GENERAL, PIPE_256, PIPE_128, PIPE_64, TINY, FEW = 0, 1, 6, 7, 16, 17

# name: (dtype, dtypeD, layoutB, group sizes, N, K, pad between rows, kernel, rows of a tile)
GROUPED = {
    "few rows, 16": ("bf16", "bf16", "k_contig", [1, 0, 3, 2, 17, 1, 0, 2], 512, 1024, 0, FEW, 16),
    "few rows, 32": ("bf16", "f32", "k_contig", [20, 9], 4096, 1024, 0, FEW, 32),
    "few rows, f16, long K": ("f16", "f16", "k_contig", [3, 2], 64, 8192, 0, FEW, 16),
    "64 x 128": ("bf16", "bf16", "k_contig", [70, 50, 128, 90, 1], 640, 1024, 0, PIPE_64, 64),
    "64 x 128, B stored K x N": ("f16", "f32", "mn_contig", [3, 0, 5, 2], 512, 512, 8, PIPE_64, 64),
    "128 x 128": ("bf16", "bf16", "k_contig", [500, 300, 0, 1, 255, 700, 129], 2048, 256, 0, PIPE_128, 128),
    "128 x 128, B stored K x N": ("f16", "f16", "mn_contig", [400, 300, 513, 720], 2048, 256, 0, PIPE_128, 128),
    "256 x 256": ("bf16", "bf16", "k_contig", [900, 1, 1300, 250, 700, 945], 2048, 512, 0, PIPE_256, 256),
    "256 x 256, B stored K x N": ("f16", "f32", "mn_contig", [1000, 1, 1200, 257, 700, 938], 2048, 512, 0, PIPE_256, 256),
    "general, 32": ("bf16", "bf16", "k_contig", [3, 7, 0, 20], 200, 130, 3, GENERAL, 32),
    "general, 64": ("f16", "f32", "mn_contig", [700, 500, 300, 400, 148], 1003, 131, 2, GENERAL, 64),
    "general, 128": ("bf16", "bf16", "k_contig", [1000, 1100, 2000, 30], 1003, 101, 3, GENERAL, 128),
    "one output per thread": ("bf16", "bf16", "k_contig", [1], 1, 5, 0, TINY, 1),
}
# name: (dtype, dtypeD, group sizes, M, N, pad, kernel, rows of a tile)
GRAD = {
    "128 x 128": ("bf16", "f32", [300, 0, 64, 1], 256, 384, 0, PIPE_128, 128),
    "256 x 256": ("f16", "f16", [100, 30, 0, 90], 2048, 2048, 0, PIPE_256, 256),
    "general, 32": ("bf16", "bf16", [30, 0, 64, 1], 70, 131, 1, GENERAL, 32),
    "general, 64": ("f16", "f32", [30, 10, 64, 1], 1000, 603, 1, GENERAL, 64),
    "general, 128": ("bf16", "f32", [30, 10, 64, 1], 2001, 603, 1, GENERAL, 128),
    "one output per thread": ("bf16", "f32", [3, 0, 9], 5, 200, 0, TINY, 1),
}
# name: (dtypeA, dtypeD, layoutA, layoutB, blockB, M, N, K, pad, kernel, rows of a tile)
F8 = {
    "few rows, 16": ("e4m3", "bf16", "k_contig", "k_contig", 128, 3, 1000, 2048, 0, FEW, 16),
    "few rows, 16, exact": ("e5m2", "f32", "k_contig", "k_contig", 128, 16, 512, 1040, 0, FEW, 16),
    "few rows, 32": ("e4m3", "bf16", "k_contig", "k_contig", 128, 30, 8192, 2048, 0, FEW, 32),
    "few rows, 64": ("e4m3", "bf16", "k_contig", "k_contig", 128, 60, 8192, 8192, 0, FEW, 64),
    "few rows, 64, exact": ("e4m3", "f16", "k_contig", "k_contig", 128, 60, 8192, 512, 0, FEW, 64),
    "64 x 128": ("e5m2", "bf16", "k_contig", "mn_contig", 128, 500, 1024, 640, 0, PIPE_64, 64),
    "64 x 128, weight gradient": ("e4m3", "f32", "mn_contig", "mn_contig", 1, 256, 384, 300, 0, PIPE_64, 64),
    "128 x 128": ("e4m3", "bf16", "k_contig", "k_contig", 128, 3000, 2048, 256, 0, PIPE_128, 128),
    "128 x 128, exact": ("e4m3", "f32", "k_contig", "mn_contig", 128, 3500, 2048, 256, 0, PIPE_128, 128),
    "128 x 128, weight gradient": ("e5m2", "bf16", "mn_contig", "mn_contig", 1, 2048, 4000, 260, 0, PIPE_128, 128),
    "256 x 256": ("e4m3", "bf16", "k_contig", "k_contig", 128, 4000, 4096, 640, 0, PIPE_256, 256),
    "256 x 256, input gradient": ("e5m2", "bf16", "k_contig", "mn_contig", 128, 4001, 4096, 512, 0, PIPE_256, 256),
    "general, 32": ("e4m3", "bf16", "mn_contig", "k_contig", 128, 200, 300, 520, 1, GENERAL, 32),
    "general, 64": ("e5m2", "f16", "k_contig", "mn_contig", 1, 1500, 2001, 260, 3, GENERAL, 64),
    "one output per thread": ("e4m3", "f32", "k_contig", "k_contig", 128, 1, 3, 9, 0, TINY, 1),
}


def operands_of_grouped(case):
    """G, M, lda, ldb, strideB as the GPU tests lay them out."""
    dt, dtD, lb, sizes, N, K, pad, kernel, tile = case
    r, c = (N, K) if lb == "k_contig" else (K, N)
    return len(sizes), sum(sizes), K + pad, c + pad, r * (c + pad)
