"""The operators around and inside the expert sublayer at the edges of their
contract on the GPU: a workspace after an error, values that are not finite,
arrays that may be the same, whole runs captured and replayed."""
import ctypes

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


# ---------------------------------------------------------------------------
# a launch that fails
# ---------------------------------------------------------------------------
def test_a_failed_launch_is_reported_by_its_own_call_alone():
    """Launches into a stream whose capture was cut short fail on the host; each call says
    so itself, and the next call, which launches nothing, does not report it again."""
    torch.zeros(1, device="cuda")                   # the primary context is current
    cu = ctypes.CDLL("libcuda.so.1")
    x, ws = filled((256,), torch.float32), moe.alloc_workspace(1 << 20)
    words = torch.zeros(2, dtype=torch.int64, device="cuda")
    p, stream, graph = x.data_ptr(), ctypes.c_void_p(), ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(stream), 1) == 0
    try:
        assert cu.cuStreamBeginCapture_v2(stream, 2) == 0
        assert cu.cuStreamSynchronize(stream) != 0          # not allowed in a capture, which it ends
        L, F = moe.lib(), moe.DTYPE_F32
        calls = {
            "norm": lambda: L.moe_layer_norm(p, F, 4, 64, 0, None, None, 1e-5, p, None, None, None, None, stream),
            "norm backward": lambda: L.moe_layer_norm_backward(p, p, F, 4, 64, 1, None, None, p, None, p, None, None,
                                                               ws.data_ptr(), ws.numel(), stream),
            "dropout": lambda: L.moe_dropout_add(p, None, F, 256, 0.5, words.data_ptr(), p, stream),
            "tiles": lambda: L.moe_quantize_tiles(p, F, 4, 64, p, p, stream),
            "product": lambda: L.moe_block_matmul(1, 16, 16, 4, None, p, p, p, p, None, F, p, ws.data_ptr(), ws.numel(),
                                                  stream),
        }
        for name, call in calls.items():
            assert call() == 4, name
            # no rows and no gradients wanted: nothing to launch
            assert L.moe_layer_norm_backward(None, None, F, 0, 64, 1, *[None] * 8, 0, None) == 0, name
    finally:
        cu.cuStreamEndCapture(stream, ctypes.byref(graph))
        assert cu.cuStreamDestroy_v2(stream) == 0
    torch.cuda.synchronize()
    assert (x == -7.0).all()


def test_both_bounded_waits_run_out():
    """The self-test goes through the wait of the layer's GEMMs and that of the block
    products: it takes the limit twice, and the error word says that both gave up."""
    ws = moe.alloc_workspace(256)
    limit_ms = 20
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    moe.moe_selftest_bounded_wait(ws, limit_ms * 1_000_000)
    end.record()
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == moe.DEVERR_WAIT_TIMEOUT
    assert start.elapsed_time(end) >= 2 * limit_ms
