"""The scoring operators where their definitions are easily lost: values that are not finite side by side, ranges of fp32,
heads with outliers, blocks of several tiles, row pointers out of order."""
import numpy as np
import pytest
import torch

from tests import test_gpu_label_logprobs as head_ops
from tests import test_gpu_logprobs as score_ops
from tests import test_gpu_q4 as q4_ops
from tests.gpu_common import need_gpu

pytestmark = pytest.mark.gpu

INF, NAN = np.inf, np.nan


# ---------------------------------------------------------------- heads
@pytest.mark.parametrize("grid,L,d", [("bf16", 3000, 768), ("bf16", 20_000, 512), ("bf16", 3000, 1024), ("e4m3", 3000, 768),
                                      ("e4m3", 20_000, 768), ("e5m2", 3000, 1024)])
def test_products_that_the_tensor_cores_cut_off(grid, L, d):
    """Tensor-core sums cut every product at 2^-25 of the largest addend: one label whose score is made of one large and
    many small products just below that, and one that the small ones lower, as far apart as this can put them the wrong
    way round."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(d)
    instructions = d // 16
    big, x_small, w_small = 256.0, 1.75 * 2.0**-15, 0.140625     # their product is 0.984 2^-25 of the large one
    lift = 1.5 * instructions * 2.0**-21 * big                  # of twice as much that the cuts may add up to
    w = rng.normal(0, 0.02, (L, d))
    a, b = L - 7, 40
    w[a], w[b] = w_small, -w_small
    w[[a, b], 0] = big
    w[a, 1], w[b, 1] = 0, np.float32(lift * 2.0**9)
    x = np.full((2, d), x_small)
    x[:, 0], x[:, 1] = 1, 2.0**-9
    W, h = head_ops.head_of(elmo, w, grid)
    X = head_ops.bf16(x)
    z = X.double().cpu().numpy() @ W.double().cpu().numpy().T
    assert z[0, a] > z[0, b] and np.argmax(z[0]) == a
    idx = head_ops.run(elmo, h, X, np.zeros(3, np.int32), np.zeros(0, np.int32), 2)[3]
    one = head_ops.run(elmo, h, X, np.zeros(3, np.int32), np.zeros(0, np.int32), 1)[3]
    assert (idx == [a, b]).all() and (one == a).all()
    h.close()
