"""Vocabulary losses (rows, vocabulary, hidden) whose gradient products are cut into two launches on a device of 256 compute
units, `add` or the output beginning in the middle of a matrix in the second.  tests/test_vocab_product_rounds.py asserts the cuts; the GPU tests
run them."""

# size: (pieces that its workspace is asked for, columns of a piece, rows of dx's first launch, columns of dw's), either mode
CUT = {(16500, 5000, 1024): (2, 2560, 16384, 2560), (2047, 8190, 2064): (1, 8190, 2047, 7168)}

# size: (workspace, columns of a piece, parts that share dx's K), either mode: several pieces whose products are split as well
SPLIT = {(40, 60000, 128): (8 << 20, 30208, 28), (100, 30011, 1040): (6 << 20, 15104, 4)}
