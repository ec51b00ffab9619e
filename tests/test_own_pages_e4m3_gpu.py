"""The own keys of the attention step over a cache in 8 bits where a part has more pages than are read at a time
(32), with the tolerances of tests/test_decode_e4m3_gpu.py."""
import pytest
import torch

import test_decode_e4m3_gpu as base
from test_decode_e4m3_gpu import built  # noqa: F401  (the build, before anything here)

pytestmark = pytest.mark.gpu


def test_many_responses_with_many_small_pages():
    # as many responses and heads as fill the GPU: parts of up to 1000 keys in pages of 16
    olens = [0, 1, 511, 512, 513, 1000, 1023, 1025, 2000, 2016]
    p = base.problem([40], [180], [olens[i % 10] if i < 170 else 33 * i % 2016 for i in range(180)], 8, 8, 64, 16,
                     torch.bfloat16, seed=1)
    base.check(p, *base.run(p), True)


@pytest.mark.parametrize("d", [64, 128])
def test_few_long_responses_with_small_pages(d):
    # more than 64 pages a part: the pages read ahead move on twice
    p = base.problem([0], [2], [17000, 16391], 2, 1, d, 16, torch.bfloat16, seed=2)
    base.check(p, *base.run(p), True)
