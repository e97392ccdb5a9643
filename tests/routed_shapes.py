"""Batches of logits whose histories are sorted by slices first (rules.hip: 128 rows and
more, 65536 and more of slices times tokens): rows, columns, tokens, biases, and the
columns of a slice."""
SHAPES = [(130, 20000, 7000, 9, 2048), (128, 9000, 14000, 3, 2048), (128, 2049, 32768, 1, 2048), (600, 3000, 33000, 5, 2048),
          (130, 40000, 8000, 7, 4096), (300, 30000, 9000, 4, 4096), (1024, 4000, 65600, 2, 4096), (260, 20011, 14000, 40, 4096)]
