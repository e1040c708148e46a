"""The operators around and inside the expert sublayer at the edges of their
contract on the GPU: a workspace after an error, values that are not finite,
arrays that may be the same, whole runs captured and replayed."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_mixture_experts_selection_b200 as moe
import sublayer_reference as ref
from sublayer_reference import blocks
from test_gpu_sublayer_ops import (CODE, TORCH, check_matmul, codes_of, dev, ffn_weights, filled, host, norm_inputs, operands,
                                   rounded, run_norm)

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


# ---------------------------------------------------------------------------
# values that are not finite
# ---------------------------------------------------------------------------
# (rows, columns) that reach each form: rows walked by resident blocks (of 4, 16 and 32 warps), a block per
# row of whole vectors, a row in several warps without them, eight rows a block
FORMS = [(600, 1024), (600, 7168), (597, 16384), (70, 2048), (40, 1001), (50, 96)]
TILED = [(600, 1024), (600, 7168), (70, 2048), (50, 96)]


def all_but(n, i):
    return [j for j in range(n) if j != i]


@pytest.mark.parametrize("shape", FORMS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", [moe.NORM_LAYER, moe.NORM_RMS])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_norm_of_a_row_that_is_not_finite(shape, dtype, kind, bad):
    """Such a row gives what the definition gives (an infinite mean square scales the
    finite values to 0), and no other row notices."""
    n, d = shape
    x, gamma, _, _ = norm_inputs(n, d, dtype, 30)
    clean = run_norm(dev(x, TORCH[dtype]), dtype, kind, dev(gamma), None)
    at = n - 2
    x[at, d - 3] = bad
    out, mean, rstd, _, _ = run_norm(dev(x, TORCH[dtype]), dtype, kind, dev(gamma), None)
    keep = all_but(n, at)
    for a, b in zip((out, mean, rstd), clean):
        assert torch.equal(a[keep], b[keep])
    with np.errstate(invalid="ignore"):
        y, m, r = ref.norm(x[at:at + 1], kind == moe.NORM_LAYER, gamma)
    assert np.array_equal(host(out)[at:at + 1], y, equal_nan=True)
    assert np.array_equal(host(mean)[at:at + 1], m, equal_nan=True)
    assert np.array_equal(host(rstd)[at:at + 1], r, equal_nan=True)


@pytest.mark.parametrize("shape", TILED)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_norm_tiles_of_a_row_that_is_not_finite(shape, dtype, bad):
    """The e4m3 copy stays the quantized output bit for bit: NaN has the code of NaN."""
    n, d = shape
    x, _, _, _ = norm_inputs(n, d, dtype, 31)
    x[n - 1, 5] = bad
    out, _, _, codes, scales = run_norm(dev(x, TORCH[dtype]), dtype, moe.NORM_RMS, None, None, tiles=True)
    c, s = torch.empty_like(codes), torch.empty_like(scales)
    moe.moe_quantize_tiles(out, CODE[dtype], n, d, c, s)
    assert torch.equal(c, codes) and torch.equal(s, scales)
    nan = torch.isnan(out)
    assert nan.sum() == (d if np.isnan(bad) else 1)
    assert torch.equal((codes & 0x7F) == 0x7F, nan) and torch.isfinite(scales).all()


@pytest.mark.parametrize("shape", FORMS + [(300, 64), (2500, 200)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", [moe.NORM_LAYER, moe.NORM_RMS])
def test_norm_backward_of_values_that_are_not_finite(shape, dtype, kind):
    """A NaN of x or dy stays in its row of dx and its column of dgamma and dbeta, one of
    dres in its value; dx may be dres itself."""
    n, d = shape
    layer, T = kind == moe.NORM_LAYER, TORCH[dtype]
    x, gamma, _, rng = norm_inputs(n, d, dtype, 32)
    dy, dres = rounded(rng.normal(size=(n, d)), dtype), rounded(rng.normal(size=(n, d)), dtype)
    _, m, r = ref.norm(x, layer)
    m, r = dev(m) if layer else None, dev(r)
    ws = moe.alloc_workspace(moe.moe_layer_norm_backward_workspace_size(n, d))

    def run(dy, x, dres):
        dx, dg, db = dev(dres, T), filled((d,), torch.float32), filled((d,), torch.float32)
        moe.moe_layer_norm_backward(dev(dy, T), dev(x, T), CODE[dtype], n, d, kind, dev(gamma), m, r, dx, dx, dg, db, ws)
        other = filled((n, d), T)
        moe.moe_layer_norm_backward(dev(dy, T), dev(x, T), CODE[dtype], n, d, kind, dev(gamma), m, r, dev(dres, T), other,
                                    None, None, ws)
        assert torch.equal(torch.nan_to_num(dx, 1e30), torch.nan_to_num(other, 1e30))
        return dx, dg, db

    clean = run(dy, x, dres)
    assert all(torch.isfinite(t).all() for t in clean)
    row, col = n - 2, d - 2
    keep_row, keep_col = all_but(n, row), all_but(d, col)
    for name in ("x", "dy", "dres"):
        arrays = {"dy": dy, "x": x, "dres": dres}
        arrays[name] = arrays[name].copy()
        arrays[name][row, col] = np.nan
        dx, dg, db = run(**arrays)
        assert torch.equal(dx[keep_row], clean[0][keep_row])
        assert torch.equal(dg[keep_col], clean[1][keep_col]) and torch.equal(db[keep_col], clean[2][keep_col])
        if name == "dres":
            assert torch.isnan(dx[row, col]) and torch.equal(dx[row, keep_col], clean[0][row, keep_col])
        else:
            assert torch.isnan(dx[row]).all()
        assert bool(torch.isnan(dg[col])) == (name != "dres")
        assert bool(torch.isnan(db[col])) == (name == "dy")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantizers_give_nan_its_code(dtype):
    """A NaN takes the code of NaN and does not count in its tile's or block's maximum."""
    rng = np.random.default_rng(33)
    n, c = 300, 272
    x = rounded(rng.normal(size=(n, c)), dtype)
    at = rng.random((n, c)) < 0.01
    at[7, 128:256] = True                           # a tile of nothing else: scale 1
    dirty = np.where(at, np.float32(np.nan), x)
    zero = np.where(at, np.float32(0), x)
    for name, args, sh in (("moe_quantize_tiles", (n, c), (n, blocks(c))),
                           ("moe_quantize_blocks", (1, n, c), (1, blocks(n), blocks(c)))):
        got = []
        for v in (dirty, zero):
            codes, scales = filled((n, c), torch.uint8, 0x55), filled(sh, torch.float32)
            getattr(moe, name)(dev(v, TORCH[dtype]), CODE[dtype], *args, codes, scales)
            got.append((codes.cpu().numpy(), host(scales)))
        (codes, scales), (want, want_s) = got
        assert np.array_equal(scales, want_s)
        assert ((codes & 0x7F) == 0x7F)[at].all() and np.array_equal(codes[~at], want[~at])
    assert not ((want & 0x7F) == 0x7F).any()


@pytest.mark.parametrize("rows,d,f", [([5, 30, 1], 272, 208), ([40, 130, 3], 272, 208), ([1], 2048, 640),
                                      ([2100, 1100], 2320, 1168)])
def test_block_ffn_of_nan_codes(rows, d, f):
    """A NaN in a row of x stays in that row, one in the gate or up weights in its expert's
    rows, one in the down weights in its column of them: short and long row tiles, a
    reduction cut into ranges, CTA pairs."""
    rng = np.random.default_rng(34)
    offsets = np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)
    R, g = int(offsets[-1]), len(rows)
    x, xs = ref.quantize_tiles(rounded(rng.normal(size=(R, d)), "bf16"))
    W = ffn_weights(rng, g, d, f)
    C = [codes_of(W[0][0]), codes_of(W[1][0]), codes_of(W[2][0])]
    S = [dev(W[i][1]) for i in range(3)]
    xc, xsd, off = codes_of(x), dev(xs), dev(offsets, torch.int32)
    ws = moe.alloc_workspace(moe.moe_block_ffn_workspace_size(g, d, f, R))

    def run(xc, C):
        out = filled((R, d), torch.float32)
        moe.moe_block_ffn(g, d, f, R, off, xc, xsd, C[0], S[0], C[1], S[1], C[2], S[2], None, moe.DTYPE_F32, out, ws)
        torch.cuda.synchronize()
        assert moe.moe_get_device_error(ws) == 0
        return out

    clean = run(xc, C)
    assert torch.isfinite(clean).all()
    bad = xc.clone()
    bad[R - 1, d - 9] = 0x7F
    out = run(bad, C)
    assert torch.isnan(out[R - 1]).all() and torch.equal(out[:R - 1], clean[:R - 1])
    e = g - 1                                       # the last expert's rows
    mine = slice(int(offsets[e]), R)
    for k in range(2):
        B = [c.clone() for c in C]
        B[k][e, f - 1, 3] = 0xFF
        out = run(xc, B)
        assert torch.isnan(out[mine]).all() and torch.equal(out[:mine.start], clean[:mine.start])
    B = [c.clone() for c in C]
    B[2][e, d - 1, f - 1] = 0x7F
    out = run(xc, B)
    assert torch.isnan(out[mine, d - 1]).all() and torch.equal(out[mine, :d - 1], clean[mine, :d - 1])
    assert torch.equal(out[:mine.start], clean[:mine.start])
