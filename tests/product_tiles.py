"""Sizes at which the layer's products run by tiles of 256 rows: at least nine steps of the contraction and a remainder, in the
last tile of either side rows and columns that are not there."""

# M, N, K of e4m3 products to bf16 (every kind of scales)
MATMUL = [(4101, 2001, 1168), (2050, 4090, 1296)]
# rows, K, F of the e4m3 block to bf16
FFN8 = [(4101, 1168, 1001)]
# rows, K, F of the bf16 block: its forward (and gate and up computed again), dx, the weights' gradients
FORWARD = [(4101, 600, 1001)]
DX = [(4101, 2000, 331)]
DW = [(601, 2000, 2101)]
