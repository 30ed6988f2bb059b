"""The epilogue of the experts' tile kernels (CPU only: compiles the kernel file to gfx950 assembly).  It moves the
accumulators of each row tile of 16 slots to LDS once: 4 writes a row tile, 16 NB in the body of NB blocks of 64 slots.  More
would be row tiles that the body does not have (an index past its accumulators), fewer rows that are lost."""
import re

import pytest

from test_expert_asm_hazards import kernels  # noqa: F401 (the fixture)


@pytest.mark.parametrize("out,write", [("t", "ds_write_b64"), ("f", "ds_write_b128")])
@pytest.mark.parametrize("blocks", [1, 4])
def test_every_row_tile_is_written_once(kernels, out, write, blocks):  # noqa: F811
    found = [lines for name, lines in kernels.items() if re.search(r"Li\dE%sLi%dEEEv" % (out, blocks), name)]
    assert len(found) == 2  # one for each format of A
    for lines in found:
        writes = sum(bool(re.match(r"\s*%s\b" % write, l)) for l in lines)
        assert writes == sum(16 * nb for nb in range(1, blocks + 1))
