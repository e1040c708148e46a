"""The operators around and inside the expert sublayer at the edges of their
contract on the GPU: a workspace after an error, values that are not finite,
arrays that may be the same, whole runs captured and replayed."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_selection_b200 as moe
from test_gpu_sublayer_ops import check_matmul, codes_of, dev, filled, operands

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# a workspace after an error
# ---------------------------------------------------------------------------
def test_clear_device_error_resets_the_control_block():
    """A call that gave up leaves the counters of the reductions it cut part-way in
    the workspace's control block; after moe_clear_device_error the next cut product
    starts from zero, in that call and the ones behind it."""
    rng = np.random.default_rng(200)
    rows, n, k = 3, 1500, 7168                      # 6 tiles of transposed rows, cut into 8 ranges
    v, s = operands(rng, rows, k)
    w, wsc = operands(rng, n, k, 1)
    x, xs, wc, wsd = codes_of(v), dev(s), codes_of(w), dev(wsc)
    ws = moe.alloc_workspace(moe.moe_block_matmul_workspace_size(1, n, k, rows))
    stale = rng.integers(1, 8, size=256).astype(np.uint8)      # counters of every tile, and the error word
    ws[:256].copy_(torch.from_numpy(stale))
    assert moe.moe_get_device_error(ws) != 0
    moe.moe_clear_device_error(ws)
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == 0
    assert not ws[:256].any()
    for _ in range(2):
        out = filled((rows, n), torch.float32)
        moe.moe_block_matmul(1, n, k, rows, None, x, xs, wc, wsd, None, moe.DTYPE_F32, out, ws)
        torch.cuda.synchronize()
        assert moe.moe_get_device_error(ws) == 0 and not ws[:256].any()
        check_matmul(out, v, s, w, wsc, [0, rows], "f32")


def test_clear_device_error_of_a_lone_word():
    """An error word that is no workspace (it does not begin on 256 bytes) is zeroed by itself."""
    words = torch.full((128,), 7, dtype=torch.int32, device="cuda")
    moe.moe_clear_device_error(words[1:2])
    torch.cuda.synchronize()
    assert words.tolist() == [7, 0] + [7] * 126
