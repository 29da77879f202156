"""The example's attention block end to end: ternary projections, rotation, paged
cache, prompt parts and decoding steps, against the block in 64 bits.

Tolerance (relative 2-norm of the last step's output, 2 sequences x 5120).  The
roundings on the way, each independent and relative to what it rounds: qkv to
bf16 and q to bf16 (2^-9 rms each, below 0.0023 through the scores and values),
keys and values to 16 bits or codes (rms 0.0023 bf16, 0.01 int8, 0.026 e4m3 of a
head's values with normal entries), weights and outputs to 16 bits (0.0023
each).  A key's error moves a score by its relative size times the score
(of unit size here) and so a weight by as much; value errors average like the
values do.  So the sum is below 2.5 x the cache's own rounding + 0.01."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from conftest import ROOT  # noqa: E402

sys.path.insert(0, os.path.join(ROOT, "examples"))
import attention_block  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache,rounding", [("x16", 0.0023), ("i8", 0.01), ("e4m3", 0.026)])
def test_attention_block(cache, rounding):
    lines = []
    err = attention_block.run(seqs=2, prompt=330, part=200, steps=3, cache=cache, out=lines.append)
    assert len(lines) == 2 + 3 + 1
    assert err <= 2.5 * rounding + 0.01
