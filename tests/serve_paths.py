"""Shapes that take each way through the 8-bit products and the mixture of
experts (test infrastructure): test_serve_paths.py holds them to the planner on
the CPU, and test_gpu_serve_paths.py runs them."""

# 8-bit products in large tiles with the rest in small ones: M, N, K, gated, what is cut
I8_CUTS = [(1794, 8780, 64, False, "columns"), (2319, 8071, 64, False, "rows"), (915, 8321, 100, True, "columns"),
           (1793, 5244, 264, True, "rows")]

# the longest K by the kernel for few tokens: one block of sixteen tokens, two and four; M, N, gated
I8_LONGEST = [(3, 4, True), (20, 4, True), (50, 4, True), (3, 8192, False), (20, 4096, False)]
LONGEST = (1 << 17) - 16

# M, D, F, E, top_k, and (blocks of 16 rows, waves) of the gated blocks and of the second products
MOE = [((1, 256, 200, 8, 2), (1, 8), (1, 8)), ((37, 2050, 301, 60, 4), (1, 4), (1, 4)), ((30, 128, 96, 12, 4), (2, 8), (2, 8)),
       ((64, 2100, 1050, 8, 2), (2, 4), (4, 4)), ((64, 2100, 1050, 16, 2), (1, 4), (2, 4)), ((64, 1000, 700, 2, 1), (4, 4), (4, 4))]
