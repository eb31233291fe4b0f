"""Sizes that run every kernel of the operators, with the tiling that each is to run in: the GPU
tests take the sizes, a CPU test asks the library's own choice for them.

Tilings: 0 256 x 256; 1 128 x 128; 2 the same with two teams of waves; 3 64 x 64 with two teams;
4 with four; -1 the kernel for few rows."""

# (m, n, k), tiling of the 8-bit product (the same with scales by rows and by tiles)
PRODUCTS = [
    ((16, 100, 1153), -1),
    ((17, 100, 1153), 4),
    ((64, 1000, 2200), 4),          # a batch of single tokens
    ((333, 3610, 1153), 3),
    ((1001, 2560, 1153), 2),
    ((2001, 2560, 1153), 1),
    ((3601, 2560, 1153), 0),
]

# (rows, d, f), tilings of the forward pass, of dx and of both dw, parts of dx
GATED = [
    ((16, 1001, 777), -1, 4, 3, 1),
    ((64, 1001, 4097), 4, 4, 0, 8),
    ((65, 999, 777), 4, 4, 3, 1),
    ((333, 1003, 4099), 2, 4, 0, 2),
    ((333, 100, 1000), 3, 4, 3, 2),
    ((777, 700, 300), 4, 4, 4, 1),
    ((1100, 700, 2080), 1, 4, 2, 1),
    ((777, 2560, 2080), 2, 2, 0, 1),
    ((1606, 1024, 4096), 0, 3, 1, 1),
    ((1606, 2560, 10240), 0, 1, 0, 1),
    ((4099, 2565, 1001), 0, 0, 1, 1),
]

# depths at which each of the four waves of the kernels for few rows runs its loop over four
# steps of 128 bytes: not at all (and three single steps), once, once and three single steps,
# several times, and with a last step that is not whole
FEW_GATED_D = [800, 1024, 1600, 4096, 4100]
FEW_PRODUCT_K = [1600, 2048, 3400, 4093, 8192]
