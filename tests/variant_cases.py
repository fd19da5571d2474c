"""Sizes that reach every kernel the product, the norm and their gradients have,
with more work a workgroup than one turn of its loops. tests/test_variants.py
runs them against 64-bit forms and shows, on the host, which kernels they take."""

# (M, N, K) of the product, plain; both formats of A. The few-lines kernels by
# lines of A, then K by what a wave has of it: part of a unit, pairs of units,
# whole quads, several quads.
GEMM = [(20, 66, 33), (32, 130, 1025), (17, 70, 2048), (32, 66, 2049), (20, 130, 4097), (32, 100, 9001),
        (5, 300, 9001), (16, 300, 20000), (1, 8300, 8193), (16, 8300, 20000), (2, 9000, 1000),
        (33, 130, 33), (64, 300, 1000), (100, 300, 5000), (40, 200, 9001), (256, 4100, 1000), (250, 4130, 5000),
        (2605, 6401, 577), (2605, 6401, 1111), (4097, 4100, 5000)]
# gated: N gate and N up lines
GATED = [(20, 33, 33), (32, 65, 1025), (17, 40, 2048), (32, 33, 2049), (20, 66, 4097), (32, 50, 9001),
         (1, 1100, 8193), (16, 1100, 20000), (5, 70, 9001), (33, 66, 33), (64, 150, 1000), (100, 150, 5000),
         (256, 4100, 1000), (250, 2100, 5000), (2605, 3203, 577), (2605, 3203, 1111), (2600, 3203, 5000)]

# (M, K) of the norm's gradient: several rows a workgroup in every kernel
NORM_BWD = [(2100, 96), (2100, 480), (2100, 1001), (2100, 2048), (2100, 2881), (2100, 4096), (1100, 5003), (1100, 8192),
            (600, 8200), (600, 16384), (600, 28672), (600, 32768), (520, 32776)]
NORM = [(300, 96), (300, 512), (300, 2048), (300, 2881), (300, 8192), (300, 16384), (50, 32768), (50, 32776)]
ACT = [(2100, 520), (4097, 2881)]
