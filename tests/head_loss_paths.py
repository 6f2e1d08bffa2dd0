"""Sizes of the head's loss that take each of its paths, and the path each takes: the tile of
the forward pass's logits, of P's (first and last piece of the vocabulary), of dW's product
(the same) and of dx's, the pieces, and the parts of dx's reduction (first and last piece).
tests/test_head_loss_paths_cpu.py holds them to the library's plan, tests/test_gpu_head_loss_paths.py
runs them.  Rows, widths and vocabularies end inside a tile and a stage."""

PATHS = {
    # name: (rows, cols, vocab), forward, P, dW, dx, pieces, parts
    "256 x 256 throughout, dx in parts": ((1675, 1736, 8916), "wide", "wide", "wide", "wide", 1, (5, 5)),
    "dx straight out of 256 x 256 tiles": ((21328, 696, 543), "wide", "wide", "mid", "wide", 1, (1, 1)),
    "three pieces in one part, as the M.1 batch": ((13037, 864, 25318), "wide", "wide", ("wide", "mid"), "wide", 3, (1, 1)),
    "three pieces in two parts, as the XS.2 batch": ((8128, 928, 37018), "wide", ("wide", "mid"), ("wide", "mid"), "wide", 3,
                                                     (2, 2)),
    "a last piece of fewer parts": ((13789, 136, 9529), "mid", "mid", "mid", "wide", 2, (4, 1)),
    "dW alone in 256 x 256 tiles": ((820, 136, 50577), "mid", "mid", "wide", "mid", 1, (36, 36)),
    "the logits alone in 256 x 256 tiles": ((150, 728, 50874), "wide", "wide", "mid", "mid", 1, (42, 42)),
    "few rows, two pieces, dx in 256 x 256 tiles and many parts": ((146, 208, 707571), "mid", "mid", "mid", "wide", 2, (256, 136)),
    "three pieces in 128 x 128 tiles and one part": ((33740, 8, 17687), "mid", "mid", "mid", "mid", 3, (1, 1)),
    "two pieces in 128 x 128 tiles and many parts": ((68, 8, 1048727), "mid", "mid", "mid", "mid", 2, (512, 3)),
    "two pieces in 32-row tiles": ((17, 8, 2227829), "rows32", "rows32", "mid", "rows32", 2, (512, 512)),
    "two pieces in 64-row tiles": ((34, 8, 2347659), "rows64", "rows64", "mid", "rows64", 2, (512, 512)),
    "one piece in 32-row tiles, one part": ((31, 72, 1000), "rows32", "rows32", "mid", "rows32", 1, (1, 1)),
    "one piece in 64-row tiles, parts": ((63, 200, 9001), "rows64", "rows64", "mid", "rows64", 1, (9, 9)),
}
