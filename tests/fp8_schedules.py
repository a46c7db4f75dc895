"""Shapes (M, N, K) of the 8-bit linear and the schedule each is for: (rows of x, rows of W per tile, CTAs
that share a tile). A rule that moves a shape elsewhere fails test_fp8_plan.py, so that the GPU tests
over these shapes keep reaching every path."""
SCHEDULES = {
    (1, 1500, 32): (16, 128, 1),          # one block: the direct store behind a single hand-over
    (1, 32000, 3840): (16, 128, 1),       # 30 blocks to one CTA: the ring goes round before the direct store
    (9, 1000, 40960): (16, 128, 8),       # 40 blocks a range: a second chunk of scales (32 blocks)
    (20, 32000, 3840): (32, 128, 1),      # 30 blocks, two chunks of 16
    (20, 1000, 20480): (32, 128, 8),      # 20 blocks a range, two chunks
    (40, 3840, 10240): (64, 128, 8),      # 10 blocks a range, two chunks of 8
    (300, 300, 384): (128, 128, 1),       # one round
    (7, 40000, 384): (128, 128, 1),       # three rounds
    (4400, 2567, 160): (128, 128, 1),     # five, a partial last block, rows that TMA cannot store
    (1089, 3840, 640): (128, 256, 1),     # one round
    (1100, 7688, 1024): (128, 256, 1),    # two
    (1100, 7693, 640): (128, 256, 1),     # two, rows that TMA cannot store
    (4096, 10240, 512): (256, 256, 2),    # nine rounds of pairs, TMA stores from three buffers in turn
    (2600, 5001, 416): (256, 256, 2),     # three, rows that TMA cannot store, a partial last block
}
