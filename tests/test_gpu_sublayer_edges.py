"""The operators around and inside the expert sublayer at the edges of their
contract on the GPU: a workspace after an error, values that are not finite,
arrays that may be the same, whole runs captured and replayed."""
import ctypes

import numpy as np
import pytest
import torch

import moe_inputs as mi
import sparse_mixture_experts_selection_b200 as moe
import sublayer_reference as ref
from sublayer_reference import U32, blocks, half_step
from test_gpu_sublayer_ops import (CODE, TORCH, check_matmul, close, codes_of, dev, ffn_weights, filled, host, norm_inputs,
                                   operands, rounded, run_norm, small_layer)

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


# ---------------------------------------------------------------------------
# captured and replayed
# ---------------------------------------------------------------------------
def captured(step):
    """A graph of the calls of step, made once before."""
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    return graph


def test_serving_sublayer_captured_and_replayed():
    """norm with its e4m3 copy, routing, the gather of codes and scales, routed and shared
    block-scaled experts and the combine as one graph: replays with new rows give what
    the calls give."""
    w, W, _ = small_layer()
    T, d, f, fs, E, K = w.T, w.d_model, w.d_ffn, w.d_ffn_shared, w.E_r, w.K
    rng = np.random.default_rng(72)
    BF = torch.bfloat16
    cfg = moe.config_for(w)
    ws = moe.alloc_workspace(moe.moe_workspace_size(cfg))
    wf = moe.alloc_workspace(max(moe.moe_block_ffn_workspace_size(E, d, f, T * K),
                                 moe.moe_block_ffn_workspace_size(1, d, fs, T)))
    D = {}
    for k, v in W.items():
        n, r, c = v.shape
        D[k] = (filled((n, r, c), torch.uint8, 0), filled((n, blocks(r), blocks(c)), torch.float32))
        moe.moe_quantize_blocks(dev(v, BF), moe.DTYPE_BF16, n, r, c, *D[k])
    x, gamma = filled((T, d), BF), dev(rng.uniform(0.5, 1.5, size=d))
    e, b = dev(mi.gen_centroids(w)), dev(mi.gen_bias(w))
    h, codes, scales = filled((T, d), BF), filled((T, d), torch.uint8, 0), filled((T, blocks(d)), torch.float32)
    i32 = lambda *sh: filled(sh, torch.int32, -5)  # noqa: E731
    idx, gates, counts = i32(T, K), filled((T, K), torch.float32), i32(E)
    off, tok, row_of, kept, rg = i32(E + 1), i32(T * K), i32(T, K), i32(E), filled((T * K,), torch.float32)
    cp, sp = filled((T * K, d), torch.uint8, 0), filled((T * K, blocks(d)), torch.float32)
    slot, shared, y = filled((T * K, d), BF), filled((1, T, d), BF), filled((T, d), BF)

    def step():
        moe.moe_layer_norm(x, moe.DTYPE_BF16, T, d, moe.NORM_RMS, gamma, None, 1e-6, h, None, None, codes, scales)
        moe.moe_route(cfg, h, e, b, None, None, idx, gates, counts, ws)
        moe.moe_permute(cfg, idx, gates, None, off, tok, row_of, kept, rg, None, ws)
        moe.moe_gather_rows(codes, T, d, tok, T * K, cp)
        moe.moe_gather_rows(scales, T, 4 * blocks(d), tok, T * K, sp)
        moe.moe_block_ffn(E, d, f, T * K, off, cp, sp, *D["gate"], *D["up"], *D["down"], rg, moe.DTYPE_BF16, slot, wf)
        moe.moe_block_ffn(1, d, fs, T, None, codes, scales, *D["sgate"], *D["sup"], *D["sdown"], None, moe.DTYPE_BF16,
                          shared, wf)
        moe.moe_combine(cfg, x, slot, shared, row_of, y)

    fresh = lambda: x.copy_(dev(rng.normal(size=(T, d)) * 3.0, BF))  # noqa: E731
    fresh()
    graph = captured(step)
    seen = []
    for _ in range(3):
        fresh()
        y.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        seen.append((y.clone(), idx.clone()))
        for t in (y, slot, shared):
            t.fill_(-7.0)
        step()
        torch.cuda.synchronize()
        assert torch.equal(y, seen[-1][0]) and torch.equal(idx, seen[-1][1])
    assert not torch.equal(seen[0][0], seen[1][0]) and torch.isfinite(seen[0][0]).all()
    assert moe.moe_get_device_error(wf) == 0 and moe.moe_get_device_error(ws) == 0


def test_cta_pairs_captured_and_replayed():
    """A product and experts on CTA pairs (launched as clusters) as one graph; the replay's
    offsets are others than the capture's."""
    rng = np.random.default_rng(73)
    n, k, R = 4400, 384, 2048
    v, s = operands(rng, R, k)
    w, wsc = operands(rng, n, k, 1)
    args = [codes_of(v), dev(s), codes_of(w), dev(wsc)]
    d, f, Rf = 2320, 1168, 4101
    W = [(codes_of(a), dev(b)) for a, b in ffn_weights(rng, 2, d, f)]
    xq, xs = ref.quantize_tiles(rounded(rng.normal(size=(Rf, d)), "bf16"))
    xq, xs = codes_of(xq), dev(xs)
    off1, off2 = dev([0, R], torch.int32), dev([0, 3001, 4101], torch.int32)
    out, y = filled((R, n), torch.bfloat16), filled((Rf, d), torch.bfloat16)
    ws = moe.alloc_workspace(max(moe.moe_block_matmul_workspace_size(1, n, k, R),
                                 moe.moe_block_ffn_workspace_size(2, d, f, Rf)))

    def step():
        moe.moe_block_matmul(1, n, k, R, off1, *args, None, moe.DTYPE_BF16, out, ws)
        moe.moe_block_ffn(2, d, f, Rf, off2, xq, xs, *W[0], *W[1], *W[2], None, moe.DTYPE_BF16, y, ws)

    graph = captured(step)
    for a, b in (([5, 2000], [0, 1, 4101]), ([0, 2048], [100, 100, 100]), ([0, 2048], [0, 3001, 4101])):
        off1.copy_(dev(a, torch.int32)), off2.copy_(dev(b, torch.int32))
        got = []
        for go in (graph.replay, step):
            out.fill_(-7.0), y.fill_(-7.0)
            go()
            torch.cuda.synchronize()
            got.append((out.clone(), y.clone()))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        assert (out[:a[0]] == -7.0).all() and (out[a[1]:] == -7.0).all() and torch.isfinite(out).all()
        assert (y[:b[0]] == -7.0).all() and (y[b[2]:] == -7.0).all()
    assert moe.moe_get_device_error(ws) == 0


def test_two_graphs_share_a_workspace():
    """Cut products captured in two graphs with one workspace, replayed in turn, and a
    norm's backward between them: the counters are back at zero behind each."""
    rng = np.random.default_rng(74)
    ops = []
    need = moe.moe_layer_norm_backward_workspace_size(300, 512)
    for rows, n, k in ((3, 1500, 7168), (90, 700, 4096)):
        v, s = operands(rng, rows, k)
        w, wsc = operands(rng, n, k, 1)
        need = max(need, moe.moe_block_matmul_workspace_size(1, n, k, rows))
        ops.append((rows, n, k, v, s, w, wsc, [codes_of(v), dev(s), codes_of(w), dev(wsc)], filled((rows, n), torch.float32)))
    ws = moe.alloc_workspace(need)
    graphs = []
    for rows, n, k, _, _, _, _, t, out in ops:
        graphs.append(captured(lambda: moe.moe_block_matmul(1, n, k, rows, None, *t, None, moe.DTYPE_F32, out, ws)))
    x, r = dev(rng.normal(size=(300, 512))), dev(np.ones(300))
    dx, dg = torch.empty_like(x), filled((512,), torch.float32)
    for _ in range(2):
        for graph, op in zip(graphs + graphs[::-1], ops + ops[::-1]):
            op[-1].fill_(-7.0)
            graph.replay()
            moe.moe_layer_norm_backward(x, x, moe.DTYPE_F32, 300, 512, moe.NORM_RMS, None, None, r, None, dx, dg, None, ws)
            torch.cuda.synchronize()
            assert not ws[:256].any()
            check_matmul(op[-1], op[3], op[4], op[5], op[6], [0, op[0]], "f32")


# ---------------------------------------------------------------------------
# places that pass 32 bits
# ---------------------------------------------------------------------------
def test_dropout_of_more_than_2_32_values():
    """The counter and the addresses behind 2^32 values, in place."""
    n, p, seed, draw = (1 << 32) + 4099, 0.25, 77, 5
    words = torch.tensor([seed, draw], dtype=torch.int64, device="cuda")
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    moe.moe_dropout_backward(x, moe.DTYPE_BF16, n, p, words, x)
    for first in (0, (1 << 31) - 2048, (1 << 32) - 2048, n // 4 * 4 - 4096):
        got = host(x[first:first + 4096]) != 0
        assert np.array_equal(got, ref.keep_mask(seed, draw, got.size, p, first=first))
    assert bool(x[-1] != 0) == bool(ref.keep_mask(seed, draw, 3, p, first=n - 3)[-1])


def test_norm_and_tiles_of_more_than_2_32_values():
    """Rows behind the 2^32nd value, in the norm with its copy, its backward and the tile
    quantizer, are the same as those rows by themselves."""
    d = 7168
    n = (1 << 32) // d + 60
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.empty((n, d), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    gamma = torch.rand(d, generator=g, device="cuda") + 0.5
    out, rstd = torch.empty_like(x), torch.empty(n, device="cuda")
    codes, scales = torch.empty((n, d), dtype=torch.uint8, device="cuda"), torch.empty((n, blocks(d)), device="cuda")
    T = moe.DTYPE_BF16
    moe.moe_layer_norm(x, T, n, d, moe.NORM_RMS, gamma, None, 1e-6, out, None, rstd, codes, scales)
    few = slice(n - 600, n)            # enough for the same blocks that walk the rows

    def same(rows, values, what):
        assert torch.equal(rows[few], values), what

    o2, r2, c2, s2 = out[few].clone(), rstd[few].clone(), codes[few].clone(), scales[few].clone()
    for t in (o2, r2, c2, s2):
        t.zero_()
    moe.moe_layer_norm(x[few].clone(), T, 600, d, moe.NORM_RMS, gamma, None, 1e-6, o2, None, r2, c2, s2)
    same(out, o2, "out"), same(rstd, r2, "rstd"), same(codes, c2, "codes"), same(scales, s2, "scales")
    codes.zero_(), scales.zero_()
    moe.moe_quantize_tiles(out, T, n, d, codes, scales)
    same(codes, c2, "tiles"), same(scales, s2, "tile scales")
    ws = moe.alloc_workspace(moe.moe_layer_norm_backward_workspace_size(n, d))
    moe.moe_layer_norm_backward(out, x, T, n, d, moe.NORM_RMS, gamma, None, rstd, None, out, None, None, ws)
    moe.moe_layer_norm_backward(o2, x[few].clone(), T, 600, d, moe.NORM_RMS, gamma, None, r2, None, o2, None, None, ws)
    same(out, o2, "dx")


@pytest.mark.parametrize("groups,n,R", [(1, 2048, (1 << 21) + 300), (1024, 5600, 780_000)])
def test_block_matmul_of_more_than_2_32_values(groups, n, R):
    """Rows of the output behind the 2^32nd value: one group on CTA pairs, and as many
    rows in 1024 groups, 762 each, on single CTAs."""
    k = 16
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    codes = lambda *sh: torch.randint(0, 0x7F, sh, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    scales = lambda *sh: torch.rand(sh, generator=g, device="cuda") + 0.5  # noqa: E731
    x, xs, w, wsc = codes(R, k), scales(R, 1), codes(groups, n, k), scales(groups, blocks(n), 1)
    off = torch.linspace(0, R, groups + 1, device="cuda", dtype=torch.float64).to(torch.int32)
    off[0], off[-1] = 0, R
    out = torch.zeros((R, n), dtype=torch.bfloat16, device="cuda")
    ws = moe.alloc_workspace(moe.moe_block_matmul_workspace_size(groups, n, k, R))
    moe.moe_block_matmul(groups, n, k, R, off, x, xs, w, wsc, None, moe.DTYPE_BF16, out, ws)
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == 0
    few = slice(R - 300, R)
    y, size = ref.product(ref.E4M3[x[few].cpu().numpy()], host(xs[few]), ref.E4M3[w[-1].cpu().numpy()], host(wsc[-1]))
    close(host(out[few]), y, (ref.product_slack(k) + 2 * U32) * size + (half_step("bf16") + U32) * np.abs(y))
