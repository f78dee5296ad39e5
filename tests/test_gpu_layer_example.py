"""GPU: the tensor-parallel block of examples/, products, all-reduce, join and
their backward passes together, against torch's binary32 autograd."""
import pytest

from examples import tensor_parallel_block as E
from tests.gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,hidden,inner,world,p", [(1, 512, 1024, 2, 0.0), (32, 1024, 2048, 8, 0.0),
                                                         (96, 1024, 4096, 4, 0.1), (40, 200, 600, 3, 0.3)])
def test_block_matches_autograd(tokens, hidden, inner, world, p):
    note(f"block tokens={tokens} hidden={hidden} inner={inner} W={world} p={p}")
    errors = E.run(tokens, hidden, inner, world, p)
    # a value passes through at most eight roundings to bf16 (y, z, u, partial,
    # sum, h, a gradient, its sum), each 2^-8 of it at most
    assert max(errors.values()) < 8 * 2.0 ** -8, errors
