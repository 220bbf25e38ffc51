"""Shapes of logits whose rows are streamed by parts of several tiles: (groups, beams, vocabulary, candidates, tiles of a part, parts of
a row), for a tile of 8192 logits (16 bits) and of 4096 (32 bits).  Vocabularies are odd, end within a tile or just behind one, or fill
their tiles to the last place."""
import torch

WIDE = [(75, 8, 8203, 8, 2, 1), (50, 8, 32003, 13, 2, 2), (100, 8, 20011, 16, 3, 1), (100, 10, 32768, 5, 4, 1), (128, 8, 40000, 16, 5, 1),
        (125, 8, 49001, 64, 6, 1), (60, 8, 110007, 10, 7, 2), (64, 8, 128256, 16, 8, 2), (1024, 1, 65535, 3, 8, 1), (16, 64, 65536, 64, 8, 1),
        (9, 57, 131001, 31, 8, 2)]
NARROW = [(75, 8, 4111, 8, 2, 1), (50, 8, 16003, 13, 2, 2), (100, 8, 10007, 16, 3, 1), (100, 10, 16384, 5, 4, 1), (128, 8, 20000, 16, 5, 1),
          (125, 8, 24501, 64, 6, 1), (60, 8, 55007, 10, 7, 2), (64, 8, 64128, 16, 8, 2), (1024, 1, 32767, 3, 8, 1), (16, 64, 32768, 64, 8, 1),
          (9, 57, 65501, 31, 8, 2)]
STREAMED = {torch.bfloat16: WIDE, torch.float16: WIDE, torch.float32: NARROW}
