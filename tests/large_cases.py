"""Calls large enough for the kernels' large forms: attention runs of several
steps a wave, joins of more splits than one turn takes, cache rows in spans of
several quads, rope waves of several rounds.  The GPU tests run them;
test_kv_plan.py holds the host's plans to what each is for, so that a change
of plan cannot quietly take a form out of the tests."""

from collections import namedtuple

# runs of several steps: seqs x heads x (16 query heads) fill the card without splitting
Attn = namedtuple("Attn", "bits d rotated heads group page seqs max_len window")
STEPS = [Attn(bits, d, rotated, 8, 4, 16, 64, 700, 0)
         for bits in (4, 8, 16) for d, rotated in ((64, False), (128, False), (128, True), (256, False), (256, True))]
# low parts of the queries in operands of their own; two tiles of heads
STEPS += [Attn(bits, d, True, 8, group, 32, 64, 523, 0) for bits in (4, 8, 16) for d in (128, 256) for group in (12, 20)]
STEPS += [Attn(4, 128, True, 8, 5, 64, 64, 1500, 700), Attn(8, 64, False, 8, 8, 16, 64, 1500, 701),
          Attn(8, 256, True, 8, 2, 128, 64, 1100, 555), Attn(16, 128, False, 8, 4, 16, 64, 900, 511)]
# what is masked, in steps after full ones; a running reference that moves in
# most steps; unwritten rows in a run of 16 steps, in two runs of 8
MASKED = [Attn(bits, d, False, 2, 4, 32, 256, 700, window) for bits in (4, 8, 16) for d in (64, 128, 256)
          for window in (0, 333)]
MOVING = [Attn(bits, 128, False, 8, 4, 64, 64, 1500, 0) for bits in (4, 8, 16)]
UNWRITTEN = [Attn(bits, 128, False, 8, 4, 64, seqs, 2048, 0) for bits in (4, 8) for seqs in (64, 32)]
# more than one run of several steps a sequence
SPLIT_STEPS = [Attn(4, 128, True, 8, 4, 64, 32, 1901, 0), Attn(8, 64, False, 4, 4, 16, 64, 1777, 0),
               Attn(16, 128, False, 8, 4, 32, 16, 1801, 0), Attn(8, 256, True, 2, 10, 32, 64, 1555, 0),
               Attn(8, 128, True, 8, 4, 64, 64, 9001, 0)]
# joins by four waves a head that take more than one turn
JOINS = [Attn(8, 128, True, 1, 4, 64, 3, 33001, 0), Attn(4, 64, False, 1, 4, 64, 1, 40001, 0),
         Attn(8, 256, True, 1, 4, 64, 2, 12001, 0), Attn(4, 128, False, 2, 1, 16, 1, 20001, 0)]

# cache rows: tokens and heads from which a wave takes several quads
Rows = namedtuple("Rows", "bits d rotated heads tokens page")
ROWS = [Rows(bits, d, rotated, heads, tokens, 16 if bits == 8 else 64)
        for bits in (4, 8, 16)
        for d, rotated, heads, tokens in ((64, False, 9, 3301), (128, False, 5, 3303), (128, True, 8, 2055),
                                          (256, False, 3, 2741), (256, True, 2, 4107))]

# rope: heads in more than one group of rounds, some part full
Rope = namedtuple("Rope", "d rot adjacent axes heads tokens")
ROPE = [Rope(128, 128, False, 1, 37, 1701), Rope(128, 128, True, 3, 5, 8195), Rope(128, 96, False, 2, 41, 1703),
        Rope(256, 64, True, 2, 67, 1641), Rope(256, 256, False, 4, 19, 1701), Rope(64, 16, False, 1, 70, 4101)]
