"""That the shapes which are meant to be streamed are (CPU): recorded launches have parts of 2 to 8 tiles in every type, of one and of several
parts a row.  Whoever changes how rows are split finds here which shapes to change."""
import re

import pytest
import torch

from beam_shapes import STREAMED
from test_beam_launches import BeamArgs, select
from test_paged_launches import ask  # noqa: F401


@pytest.mark.parametrize("masked", (False, True))
@pytest.mark.parametrize("kind,dtype", [(0, torch.bfloat16), (1, torch.float16), (2, torch.float32)])
def test_tiles_and_parts(ask, kind, dtype, masked):  # noqa: F811
    shapes = STREAMED[dtype]
    for (G, K, V, M, tiles, parts), (ret, launches) in zip(shapes, ask([select(kind, *s[:4], allowed=0x6000 if masked else None) for s in shapes])):
        assert ret == 0
        name, grid, block, arg = launches[0]
        a = BeamArgs.from_buffer_copy(bytes.fromhex(arg))
        assert re.search(rf"k_beam_partsILi{kind}ELi4ELb{int(masked)}E", name), name
        assert (a.tiles, a.parts) == (tiles, parts), (G, K, V)
    assert {s[4] for s in shapes} == set(range(2, 9)) and {s[5] for s in shapes} == {1, 2}
