"""Shapes (rows, weight rows or features, K) that the choice of kernel sends to each
kernel: test_tile_choice.py asserts that it does, test_gpu_tile_variants.py runs
them.  A kernel is named by its tile (1000 * rows + weight rows); 0 is the kernel
for few rows."""

# int8 product, the largest K there is: no multiple of 128, 1024 chunks
I8_LARGEST_SUM = {0: (200, 140), 32064: (199, 2001), 64064: (390, 4001), 128128: (1590, 2001),
                  256128: (2999, 2010), 256256: (1590, 8001)}
I8_LARGEST_SUM_K = 131056
# int8 product and gated block (weight rows 2F): long K, one row or column more than whole tiles
I8_LONG_K = {0: (30, 1001, 7184), 32064: (193, 2049, 7184), 64064: (385, 4033, 7056),
             128128: (769, 4225, 7184), 256128: (1537, 4097, 7312), 256256: (3073, 4097, 7184)}
I8_GATED_LONG_K = {0: (30, 501, 7184), 32064: (193, 1025, 7184), 64064: (385, 2017, 7056),
                   128128: (769, 2113, 7184), 256128: (1537, 2049, 7312),
                   256256: (3073, 2049, 7184)}
# E4M3 gated block (M, F, K)
GATED_LONG_K = {0: (17, 1024, 7168), 64128: (257, 2048, 7168), 128128: (769, 2048, 7168),
                256128: (1537, 2048, 7168), 256256: (3073, 2048, 7168)}
