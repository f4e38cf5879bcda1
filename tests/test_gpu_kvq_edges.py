"""GPU: tree attention over the 8-bit cache at the ends of its envelope: more query heads a KV head than
the tcgen05 kernels take, as many groups as the entry point allows, the largest row counts."""
import pytest

from test_gpu_kvq_attn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("shape", [
    (1, 2, 4200, 1, 128, 70, [70]), (1, 1, 9000, 1, 128, 300, [290]), (1, 3, 4200, 1, 64, 70, [70]),
    (1, 32, 4096, 1, 128, 40, [33]),                # the most that the tcgen05 kernels take
    (65535, 1, 1, 1, 128, 1, [1] * 65535),          # one token over one, every group there is
    (32767, 1, 2, 2, 64, 3, [2] * 32767),
], ids=lambda s: "-".join(map(str, s[:6])))
def test_largest_shapes(shape, precise):
    c = Case(61, *shape)
    c.check(c.desc(precise, precise))
