"""Products whose sizes select a given tile shape of the dense GEMMs (csrc/gemm_shape.hpp `choose_tile`) on a device of
256 compute units.  tests/test_tile_choice.py asserts the choices, so that a change of the estimate cannot leave a
kernel untested unnoticed; the GPU tests run the products.

Shapes: 0: 256 x 256, 1: 128 x 128, 2: 64 x 128, 3: 64 x 128 with three stages of loads."""

# (M, N, K): (shape in the exact mode, on the FP8 cores), without a workspace, hence without a split of K.  M, N and K
# are ragged against every tile; N is a multiple of 16 where B may be stored [K x N].
PLAIN = {(2973, 4130, 528): (0, 0), (1990, 4106, 400): (1, 1), (1027, 908, 3808): (3, 3), (1437, 2490, 352): (1, 2),
         (300, 260, 272): (2, 3)}
PLAIN_BT = {(2973, 4144, 528): (0, 0), (1990, 4112, 400): (1, 1), (2313, 4384, 32): (1, 1), (1027, 912, 3808): (3, 3),
            (1437, 2496, 352): (1, 2), (300, 272, 272): (2, 3)}
# the largest K (a 34 GB operand each way at 256 x 256), and K N just under 2^31 for B stored [K x N]
LARGEST_K = {(3845, 4090, 1 << 23): (0, 0), (1990, 4090, 1 << 23): (1, 1)}
LARGEST_KN_BT = {(3845, 4096, (1 << 19) - 16): (0, 0), (1990, 4096, (1 << 19) - 16): (1, 1)}

WORKSPACE = 64 << 20
# (M, rows of B, K): (shape, split of K in the exact mode, on the FP8 cores) of the products with a feed-forward
# epilogue, over a workspace of WORKSPACE bytes.  The gated product has half as many output columns as rows of B.
EPILOGUE = {(1990, 4106, 400): ((1, 1), (1, 1)), (2313, 4384, 32): ((1, 1), (1, 1)), (195, 4156, 4112): ((1, 3), (1, 3)),
            (2131, 386, 4368): ((1, 3), (1, 3)), (454, 8206, 4016): ((0, 3), (0, 3)), (2973, 4132, 528): ((0, 1), (0, 1)),
            (2973, 4144, 528): ((0, 1), (0, 1)), (300, 264, 272): ((2, 1), (3, 1)), (23, 56, 736): ((2, 6), (2, 6)),
            (1969, 34, 2416): ((3, 6), (3, 6))}
