"""Vocabulary losses (rows, vocabulary, hidden) whose products select given tile shapes and cuts (csrc/gemm_rounds.hpp
`plan_rounds`) on a device of 256 compute units.  tests/test_vocab_rounds.py asserts the choices; the GPU tests run them.

Shapes as in tile_cases.py; the three-stage 64 x 128 tiles are taken as the two-stage ones by the loss's own products."""

# size: {mode (0 exact, 1 FP8 cores): (columns of the first launch, its shape, shape of the rest or None)} of the logits' product
LOGITS = {(200, 3001, 1040): {0: (3001, 3, None), 1: (3001, 3, None)}, (1023, 8190, 2064): {0: (8190, 1, None), 1: (8190, 1, None)},
          (2047, 8190, 2064): {0: (8190, 0, None), 1: (8190, 0, None)}, (2047, 8201, 2048): {0: (8192, 0, 3), 1: (8192, 0, 3)},
          (8192, 1111, 528): {0: (1111, 1, None), 1: (1111, 1, None)}}
