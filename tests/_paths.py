"""One shape for every path that computes the grouped products, with the launch
plan it is meant to take.  test_grouped_plan.py holds the plans to it on the
CPU, so that a rule that moves a shape to another path is noticed;
test_gpu_paths.py runs them."""

STREAM, T64, T128, T256 = 0, 1, 2, 3     # moe_product_kernel

# Rows products: T, topk, E, block_m, the reduction's length, the output's width
# (dx takes the same with K and N exchanged), kernel, ranges of the reduction.
ROWS = {
    "stream": (4, 2, 8, 2, 200, 40, STREAM, 1),
    "stream, quarters": (4, 2, 8, 2, 1032, 72, STREAM, 1),
    "stream, ranges": (4, 2, 8, 2, 8200, 40, STREAM, 4),
    "small": (101, 2, 3, 16, 72, 136, T64, 1),
    "small, ranges": (101, 2, 3, 16, 4096, 136, T64, 8),
    "small, odd": (101, 2, 3, 16, 73, 131, T64, 1),
    "small, narrow": (101, 2, 3, 16, 5, 7, T64, 1),
    "small, odd, ranges": (101, 2, 3, 16, 2051, 61, T64, 4),
    "128 x 128": (701, 2, 2, 16, 65, 4100, T128, 1),
    "full": (701, 2, 3, 16, 1032, 4104, T256, 1),
    "full, ranges": (1030, 1, 1, 16, 7304, 1096, T256, 4),
}

# the stream is a forward kernel
OP_PATHS = [(op, name) for op in ("fwd", "dx") for name in ROWS
            if op == "fwd" or not name.startswith("stream")]

# Weight gradients: rows of each expert (a multiple of topk in all), topk,
# block_m, K, N, kernel, ranges of an expert's rows.
DW = {
    "small": ((301, 0, 699), 2, 16, 200, 136, T64, 1),
    "small, odd": ((301, 0, 599), 2, 16, 133, 71, T64, 1),
    "small, narrow": ((301, 0, 599), 2, 16, 5, 7, T64, 1),
    "128 x 128": ((70, 391, 0, 239), 2, 16, 1030, 2051, T128, 1),
    # more than 256 tiles of up to seven steps: a workgroup stays for several,
    # and its copies run on from one into the next
    "full, many tiles": ((70, 0, 390, 129, 0, 260, 5, 346), 2, 16, 2056, 4104, T256, 1),
    "full, many tiles, two experts": ((190, 65), 1, 1, 4104, 4104, T256, 1),
    "full, ranges": ((6011, 0, 5989), 2, 16, 136, 72, T256, 4),
}


def rows_R(name):
    T, topk, E, bm = ROWS[name][:4]
    return T * topk + E * (bm - 1)


def dw_R(name, padded=True):
    counts, _, bm = DW[name][:3]
    return sum(counts) + (len(counts) * (bm - 1) if padded else 0)
