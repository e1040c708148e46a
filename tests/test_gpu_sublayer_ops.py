"""The operators around and inside the expert sublayer on the GPU against their
plain 64-bit forms (sublayer_reference), at the sizes and values where they can
go wrong.  Every tolerance is the sum of what the arithmetic allows: half a step
of the output's type for its one rounding and the bounds that the reference
derives for fp32 sums."""
import numpy as np
import pytest
import torch

import moe_inputs as mi
from oracle import moe_oracle as mo
import sparse_mixture_experts_selection_b200 as moe
import sublayer_reference as ref
from sublayer_reference import U32, blocks, half_step

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
CODE = {"f32": moe.DTYPE_F32, "bf16": moe.DTYPE_BF16}


def dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def host(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def rounded(a, dtype):
    return mi.round_bf16(a.astype(np.float32)) if dtype == "bf16" else a.astype(np.float32)


def filled(shape, dtype, value=-7.0):
    return torch.full(shape, value, dtype=dtype, device="cuda")


def close(got, want, bound):
    got, want = np.asarray(got), np.asarray(want)
    bad = np.abs(got - want) - bound
    at = np.unravel_index(int(np.argmax(bad)), bad.shape)
    assert np.all(np.isfinite(got)) and bad[at] <= 0, (at, got[at], want[at], np.broadcast_to(bound, bad.shape)[at])


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
def norm_inputs(n, d, dtype, seed, offset=1.0):
    rng = np.random.default_rng([seed, n, d])
    x = rng.normal(size=(n, d)) * np.exp(0.5 * rng.normal(size=d)) + offset * rng.normal(size=(n, 1))
    if n > 2:
        x[1] = 0.0                     # variance 0: xhat 0, rstd 1 / sqrt(eps)
        x[2] = x[2] * 1e-3 + 1000.0    # a mean far above the spread
    return rounded(x, dtype), rng.normal(size=d).astype(np.float32), rng.normal(size=d).astype(np.float32), rng


def run_norm(x, dtype, kind, gamma, beta, eps=1e-6, tiles=False, out=None):
    n, d = x.shape
    out = filled((n, d), TORCH[dtype]) if out is None else out
    mean, rstd = filled((n,), torch.float32), filled((n,), torch.float32)
    codes = filled((n, d), torch.uint8, 0x55) if tiles else None
    scales = filled((n, blocks(d)), torch.float32) if tiles else None
    moe.moe_layer_norm(x, CODE[dtype], n, d, kind, gamma, beta, eps, out, mean, rstd, codes, scales)
    return out, mean, rstd, codes, scales


# the last line: batches long enough for the blocks that walk the rows, at each of their widths
NORM_SHAPES = [(1, 1), (3, 7), (5, 8), (4, 64), (33, 100), (300, 256), (17, 1001), (9, 1024), (65, 2048), (12, 2056),
               (6, 4100), (5, 7168), (3, 8200), (3, 16383), (4, 16384), (1, 7168), (601, 16),
               (593, 520), (700, 1032), (613, 2048), (641, 5000), (597, 7168), (593, 9000), (595, 16384),
               # on both sides of the sizes from which rows are walked by resident blocks
               (443, 1024), (444, 1024), (444, 1016), (450, 512), (2, 512), (150, 504), (1, 256), (149, 256), (2100, 640)]


@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", [moe.NORM_LAYER, moe.NORM_RMS])
def test_norm(shape, dtype, kind):
    n, d = shape
    x, gamma, beta, _ = norm_inputs(n, d, dtype, kind)
    use_beta = kind == moe.NORM_LAYER or d % 2 == 0
    out, mean, rstd, _, _ = run_norm(dev(x, TORCH[dtype]), dtype, kind, dev(gamma), dev(beta) if use_beta else None)
    layer = kind == moe.NORM_LAYER
    y, m, r = ref.norm(x, layer, gamma, beta if use_beta else None)
    close(host(out), y, ref.norm_bound(x, layer, gamma, y, m, r, dtype))
    close(host(mean), m, 48 * U32 * np.abs(x.astype(np.float64)).mean(1))
    # rstd through the mean square: half its relative error, and the mean's error, which enters squared and
    # through sum(c), which vanishes
    shift = 48 * U32 * np.abs(x.astype(np.float64)).mean(1) if layer else 0.0
    close(host(rstd), r, r * (40 * U32 + 0.5 * (shift * r) ** 2 + 2 * U32 * shift * r))


def test_norm_without_gains_and_in_place():
    x, _, _, _ = norm_inputs(40, 512, "bf16", 5)
    t = dev(x, torch.bfloat16)
    want, _, _, _, _ = run_norm(t, "bf16", moe.NORM_LAYER, None, None)
    same, _, _, _, _ = run_norm(t, "bf16", moe.NORM_LAYER, None, None, out=t)
    assert torch.equal(want, same)
    y, m, r = ref.norm(x, True)
    close(host(want), y, ref.norm_bound(x, True, None, y, m, r, "bf16"))
    # a long batch of wide rows: the rows ahead are on their way while this one is written
    t = dev(norm_inputs(1500, 2048, "bf16", 6)[0], torch.bfloat16)
    want, _, _, _, _ = run_norm(t, "bf16", moe.NORM_RMS, None, None)
    same, _, _, _, _ = run_norm(t, "bf16", moe.NORM_RMS, None, None, out=t)
    assert torch.equal(want, same)


@pytest.mark.parametrize("shape", [(1, 16), (5, 128), (33, 144), (64, 2048), (7, 7168), (3, 16384), (300, 272),
                                   (700, 2048), (605, 7168), (600, 9008)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_tiles_are_the_quantized_output(shape, dtype):
    n, d = shape
    x, gamma, _, _ = norm_inputs(n, d, dtype, 11)
    out, _, _, codes, scales = run_norm(dev(x, TORCH[dtype]), dtype, moe.NORM_RMS, dev(gamma), None, tiles=True)
    q, s = ref.quantize_tiles(host(out))
    assert np.array_equal(host(scales), s)
    assert np.array_equal(codes.cpu().numpy(), ref.encode(q))
    # codes alone, without the output
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    moe.moe_layer_norm(dev(x, TORCH[dtype]), CODE[dtype], n, d, moe.NORM_RMS, dev(gamma), None, 1e-6, None, None, None,
                       c2, s2)
    assert torch.equal(c2, codes) and torch.equal(s2, scales)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_norm_keeps_bad_rows_to_themselves(bad):
    x, gamma, _, _ = norm_inputs(20, 100, "f32", 6)
    clean, _, _, _, _ = run_norm(dev(x), "f32", moe.NORM_LAYER, dev(gamma), None)
    x[4, 37] = bad
    out, mean, rstd, _, _ = run_norm(dev(x), "f32", moe.NORM_LAYER, dev(gamma), None)
    keep = [i for i in range(20) if i != 4]
    assert torch.equal(out[keep], clean[keep])
    assert not torch.isfinite(out[4]).any()


@pytest.mark.parametrize("shape", NORM_SHAPES + [(2500, 64), (1300, 328)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", [moe.NORM_LAYER, moe.NORM_RMS])
def test_norm_backward(shape, dtype, kind):
    n, d = shape
    layer = kind == moe.NORM_LAYER
    x, gamma, _, rng = norm_inputs(n, d, dtype, 20 + kind)
    dy, dres = rounded(rng.normal(size=(n, d)), dtype), rounded(rng.normal(size=(n, d)), dtype)
    _, m, r = ref.norm(x, layer, eps=1e-6)
    m, r = m.astype(np.float32), r.astype(np.float32)
    with_res, use_gamma = n % 2 == 1, d % 3 != 0
    T = TORCH[dtype]
    ws = moe.alloc_workspace(moe.moe_layer_norm_backward_workspace_size(n, d))
    dx, dg, db = filled((n, d), T), filled((d,), torch.float32), filled((d,), torch.float32)
    args = [dev(dy, T), dev(x, T), CODE[dtype], n, d, kind, dev(gamma) if use_gamma else None,
            dev(m) if layer else None, dev(r), dev(dres, T) if with_res else None]
    moe.moe_layer_norm_backward(*args, dx, dg, db, ws)
    want, wg, wb, size = ref.norm_backward(dy, x, layer, gamma if use_gamma else None, m, r, dres if with_res else None)
    close(host(dx), want, 64 * U32 * size + (half_step(dtype) + 2 * U32) * np.abs(want))
    # sums over the rows: the longest chain is a block's rows, then its share of the parts
    xhat = (x.astype(np.float64) - m[:, None] * layer) * r[:, None]
    chain = (n // 296 + 1 + 296 * 8 // 8 + 16) * U32
    close(host(dg), wg, chain * np.abs(dy * xhat).sum(0) + 1e-30)
    close(host(db), wb, chain * np.abs(dy.astype(np.float64)).sum(0) + 1e-30)
    # the same bits again, in place, and with the sums left out
    dx2, dg2, db2 = args[0].clone(), torch.empty_like(dg), torch.empty_like(db)
    moe.moe_layer_norm_backward(dx2, *args[1:], dx2, dg2, db2, ws)
    assert torch.equal(dx2, dx) and torch.equal(dg2, dg) and torch.equal(db2, db)
    dx3, dg3 = torch.empty_like(dx), torch.empty_like(dg)
    moe.moe_layer_norm_backward(*args, dx3, None, None, ws)
    moe.moe_layer_norm_backward(*args, dx3, dg3, None, ws)
    assert torch.equal(dx3, dx) and torch.equal(dg3, dg)


@pytest.mark.parametrize("kind", [moe.NORM_LAYER, moe.NORM_RMS])
def test_norm_backward_against_differences(kind):
    """The kernel's dx along a direction against differences of the 64-bit norm."""
    rng = np.random.default_rng(8)
    n, d, layer = 5, 300, kind == moe.NORM_LAYER
    x, dy, v = (rng.normal(size=(n, d)).astype(np.float32) for _ in range(3))
    gamma = rng.normal(size=d).astype(np.float32)
    out, mean, rstd, _, _ = run_norm(dev(x), "f32", kind, dev(gamma), None)
    dx = torch.empty_like(out)
    ws = moe.alloc_workspace(moe.moe_layer_norm_backward_workspace_size(n, d))
    moe.moe_layer_norm_backward(dev(dy), dev(x), moe.DTYPE_F32, n, d, kind, dev(gamma), mean, rstd, None, dx, None, None, ws)
    h = 1e-5
    f = lambda t: (ref.norm(t, layer, gamma)[0] * dy).sum(1)  # noqa: E731
    diff = (f(x + h * v.astype(np.float64)) - f(x - h * v.astype(np.float64))) / (2 * h)
    # |dx . v| sums d terms of fp32 values; the differences' own error is of order h^2
    size = (np.abs(host(dx)) * np.abs(v)).sum(1)
    close((host(dx) * v).sum(1), diff, 256 * U32 * (size + np.abs(dy * gamma * v).sum(1)) + 1e-7)


def test_norm_of_no_rows():
    dg, db = filled((64,), torch.float32), filled((64,), torch.float32)
    e = torch.empty((0, 64), device="cuda")
    ws = moe.alloc_workspace(moe.moe_layer_norm_backward_workspace_size(0, 64))
    moe.moe_layer_norm(e, moe.DTYPE_F32, 0, 64, 0, None, None, 1e-5, e)
    moe.moe_layer_norm_backward(e, e, moe.DTYPE_F32, 0, 64, 0, None, e, e, None, e, dg, db, ws)
    assert not host(dg).any() and not host(db).any()


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------
def rng_words(seed, draw):
    return torch.tensor([seed, draw], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("n", [1, 3, 4, 7, 8, 9, 1000, 4097, 1 << 20, (1 << 21) + 5])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999, 1.0])
def test_dropout(n, dtype, p):
    rng = np.random.default_rng(n)
    T = TORCH[dtype]
    x, res = rounded(rng.normal(size=n), dtype), rounded(rng.normal(size=n), dtype)
    seed, draw = 0x1234567890ABCDEF, 0x0FEDCBA987654321
    words = rng_words(seed, draw)
    out, dx = filled((n,), T), filled((n,), T)
    moe.moe_dropout_add(dev(x, T), dev(res, T), CODE[dtype], n, p, words, out)
    moe.moe_dropout_backward(dev(x, T), CODE[dtype], n, p, words, dx)
    keep = ref.keep_mask(seed, draw, n, p)
    drop = np.where(keep, x.astype(np.float64) / max(1.0 - p, 1e-9), 0.0)
    # the scale is rounded to fp32, then one fused multiply-add and the output's rounding
    tol = lambda want: 2 * U32 * np.abs(drop) + (half_step(dtype) + U32) * np.abs(want)  # noqa: E731
    close(host(dx), drop, tol(drop))
    close(host(out), drop + res, tol(drop + res))
    assert np.array_equal(host(dx) != 0, keep & (x != 0))
    same = dev(x, T)
    moe.moe_dropout_add(same, dev(res, T), CODE[dtype], n, p, words, same)
    assert torch.equal(same, out)


def test_dropout_leaves_dropped_nans_out():
    n, words = 4096, rng_words(-3, 7)                # a seed with its top bit set
    keep = ref.keep_mask((1 << 64) - 3, 7, n, 0.5)
    x = np.where(keep, 1.0, np.nan).astype(np.float32)
    out = filled((n,), torch.float32)
    moe.moe_dropout_add(dev(x), None, moe.DTYPE_F32, n, 0.5, words, out)
    assert np.array_equal(host(out), np.where(keep, 2.0, 0.0))


# ---------------------------------------------------------------------------
# quantizers
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("shape", [(1, 16), (3, 112), (5, 128), (37, 144), (300, 7168), (4097, 64), (5000, 1040)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_tiles_bit_exact(shape, dtype):
    n, c = shape
    rng = np.random.default_rng(n + c)
    x = rounded(rng.normal(size=(n, c)) * rng.choice([1e-30, 1e-3, 1.0, 600.0, 3e20], size=(n, 1)), dtype)
    x[0, :8] = rounded(np.array([-1e-38, 0.0, -0.0, 448.0, -448.0, 1e-5, 7.0, -3.5]), dtype)
    if n > 2:
        x[2] = 0.0
    codes, scales = filled((n, c), torch.uint8, 0x55), filled((n, blocks(c)), torch.float32)
    moe.moe_quantize_tiles(dev(x, TORCH[dtype]), CODE[dtype], n, c, codes, scales)
    q, s = ref.quantize_tiles(x)
    assert np.array_equal(host(scales), s)
    assert np.array_equal(codes.cpu().numpy(), ref.encode(q))


@pytest.mark.parametrize("shape", [(1, 1, 16), (3, 129, 144), (2, 300, 256), (1, 2048, 272), (5, 128, 128)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_blocks_bit_exact(shape, dtype):
    n, r, c = shape
    rng = np.random.default_rng(r + c)
    w = rounded(rng.normal(size=shape) * np.exp2(rng.integers(-20, 20, size=(n, r, 1))), dtype)
    w[0, :, :16] = 0.0
    codes = filled(shape, torch.uint8, 0x55)
    scales = filled((n, blocks(r), blocks(c)), torch.float32)
    moe.moe_quantize_blocks(dev(w, TORCH[dtype]), CODE[dtype], n, r, c, codes, scales)
    q, s = ref.quantize_blocks(w)
    assert np.array_equal(host(scales), s)
    assert np.array_equal(codes.cpu().numpy(), ref.encode(q))


# ---------------------------------------------------------------------------
# block-scaled products
# ---------------------------------------------------------------------------
def operands(rng, rows, cols, n=None):
    """Values on the e4m3 grid and scales of another rule than the quantizers' (no powers of two)."""
    shape = (rows, cols) if n is None else (n, rows, cols)
    v = ref.to_grid(np.clip(rng.normal(size=shape) * 100, -448, 448))
    sb = (rows, blocks(cols)) if n is None else (n, blocks(rows), blocks(cols))
    s = (np.exp(rng.normal(size=sb)) / 100).astype(np.float32)
    return v, s.astype(np.float64)


def codes_of(v):
    return dev(ref.encode(v), torch.uint8)


def run_matmul(v, s, w, wsc, offsets, dtype, row_scale=None, out=None, codes=None):
    g, n, k = w.shape
    rows = v.shape[0]
    out = filled((rows, n), TORCH[dtype]) if out is None else out
    ws = moe.alloc_workspace(moe.moe_block_matmul_workspace_size(g, n, k, rows))
    moe.moe_block_matmul(g, n, k, rows, None if offsets is None else dev(offsets, torch.int32),
                         codes_of(v) if codes is None else codes, dev(s), codes_of(w), dev(wsc),
                         None if row_scale is None else dev(row_scale), CODE[dtype], out, ws)
    torch.cuda.synchronize()
    return out, moe.moe_get_device_error(ws)


def check_matmul(out, v, s, w, wsc, offsets, dtype, row_scale=None):
    got = host(out)
    for g in range(w.shape[0]):
        a, b = offsets[g], offsets[g + 1]
        if a == b:
            continue
        y, size = ref.product(v[a:b], s[a:b], w[g], wsc[g])
        sc = 1.0 if row_scale is None else row_scale[a:b, None].astype(np.float64)
        close(got[a:b], y * sc, (ref.product_slack(w.shape[2]) + 2 * U32) * size * np.abs(sc)
              + (half_step(dtype) + U32) * np.abs(y * sc))


MATMULS = [  # rows of each group, n, k
    ([1], 1, 16), ([1], 128, 128), ([3, 0, 5], 130, 144), ([128], 256, 256), ([129, 0, 0, 1], 257, 272),
    ([300, 17], 255, 640), ([0, 40, 0], 96, 16), ([64] * 20, 64, 384), ([1] * 70, 33, 400), ([513], 1000, 112),
    ([31, 33, 95, 97, 127, 128, 255, 257], 384, 1024), ([1, 0] * 512, 40, 144), ([16, 17, 32, 15, 160, 144], 513, 528), ([0, 0], 64, 64), ([7], 2048, 7168), ([2, 1], 320, 4112),
    # enough rows a group and tiles for CTA pairs: whole, ragged and odd, one block of columns in the last tile
    ([2048], 4400, 384), ([1700, 29, 900], 6301, 272), ([0, 3000, 1], 4952, 912),
]


@pytest.mark.parametrize("case", range(len(MATMULS)))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_matmul(case, dtype):
    rows, n, k = MATMULS[case]
    rng = np.random.default_rng(case)
    offsets = np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)
    R = int(offsets[-1]) + 5                        # five rows behind the last group
    v, s = operands(rng, R, k)
    w, wsc = operands(rng, n, k, len(rows))
    gate = rng.uniform(0.1, 1, size=R).astype(np.float32) if case % 2 else None
    out, err = run_matmul(v, s, w, wsc, offsets, dtype, gate)
    assert err == 0
    check_matmul(out, v, s, w, wsc, offsets, dtype, gate)
    assert (host(out)[offsets[-1]:] == -7.0).all()
    again, _ = run_matmul(v, s, w, wsc, offsets, dtype, gate)
    assert torch.equal(again, out)


def test_block_matmul_without_offsets_and_first_rows_skipped():
    rng = np.random.default_rng(50)
    v, s = operands(rng, 150, 256)
    w, wsc = operands(rng, 192, 256, 1)
    out, _ = run_matmul(v, s, w, wsc, None, "f32")
    check_matmul(out, v, s, w, wsc, [0, 150], "f32")
    part, err = run_matmul(v, s, w, wsc, [20, 111], "f32")
    assert err == 0
    assert torch.equal(part[20:111], out[20:111])
    assert (host(part)[:20] == -7).all() and (host(part)[111:] == -7).all()


@pytest.mark.parametrize("rows,n,k", [([100, 7, 200], 300, 512), ([1], 200, 2048), ([2100], 4352, 1024)])
@pytest.mark.parametrize("shifted", [(1, 0), (0, 1), (3, 2)])
def test_block_matmul_scales_at_any_four_bytes(rows, n, k, shifted):
    """Scales that begin between 16-byte addresses, and NaN in the words around them,
    give the very sums that aligned ones do."""
    rng = np.random.default_rng(57)
    offsets = dev(np.concatenate([[0], np.cumsum(rows)]), torch.int32)
    R, g = sum(rows), len(rows)
    v, s = operands(rng, R, k)
    w, wsc = operands(rng, n, k, g)
    x, wc = codes_of(v), codes_of(w)
    outs = []
    for by in [(0, 0), shifted]:
        scales = []
        for a, b in zip([dev(s), dev(wsc)], by):
            room = torch.full((a.numel() + 8,), float("nan"), device="cuda")
            room[b:b + a.numel()] = a.flatten()
            scales.append(room[b:b + a.numel()].view(a.shape))
        out = filled((R, n), torch.float32)
        ws = moe.alloc_workspace(moe.moe_block_matmul_workspace_size(g, n, k, R))
        moe.moe_block_matmul(g, n, k, R, offsets, x, scales[0], wc, scales[1], None, moe.DTYPE_F32, out, ws)
        torch.cuda.synchronize()
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.isfinite(outs[0]).all()


def test_block_matmul_nan_codes_stay_in_their_rows_and_columns():
    rng = np.random.default_rng(51)
    v, s = operands(rng, 140, 384)
    w, wsc = operands(rng, 200, 384, 2)
    offsets = [0, 60, 133]
    clean, _ = run_matmul(v, s, w, wsc, offsets, "f32")
    codes = codes_of(v)
    codes[10, 200] = 0x7F                          # a NaN in a row of the first group
    codes[133:] = 0xFF                             # NaN in rows of no group
    out, err = run_matmul(v, s, w, wsc, offsets, "f32", codes=codes)
    assert err == 0
    keep = [i for i in range(133) if i != 10]
    assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[10]).all()


@pytest.mark.parametrize("offsets", [[0, 10, 41, 40], [-1, 10, 20, 40], [0, 10, 20, 41], [0, 40, 0, 40]])
def test_block_matmul_reports_bad_offsets(offsets):
    """Decreasing and too large offsets are met on the device: the error word is set
    and nothing is written."""
    rng = np.random.default_rng(52)
    v, s = operands(rng, 40, 512)
    w, wsc = operands(rng, 64, 512, 3)
    out, err = run_matmul(v, s, w, wsc, offsets, "f32")
    assert err == moe.DEVERR_INDEX
    assert (host(out) == -7).all()


# ---------------------------------------------------------------------------
# block-scaled experts
# ---------------------------------------------------------------------------
FFNS = [  # rows of each expert, d, f
    ([1], 16, 16), ([1], 256, 128), ([5, 0, 130], 144, 208), ([64, 1, 0, 33], 512, 384), ([257], 128, 1040),
    ([3] * 40, 272, 96), ([1], 2048, 640), ([0, 200, 129], 640, 272),
    ([3001, 1100], 2320, 1168),                     # both products on CTA pairs
]


def run_ffn(x, xs, W, offsets, dtype, gate, rows):
    (wg, sg), (wu, su), (wd, sd) = W
    g, f, d = wg.shape
    out = filled((rows, d), TORCH[dtype])
    ws = moe.alloc_workspace(moe.moe_block_ffn_workspace_size(g, d, f, rows))
    moe.moe_block_ffn(g, d, f, rows, None if offsets is None else dev(offsets, torch.int32), x, xs, codes_of(wg),
                      dev(sg), codes_of(wu), dev(su), codes_of(wd), dev(sd), None if gate is None else dev(gate),
                      CODE[dtype], out, ws)
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == 0
    return out


def ffn_weights(rng, g, d, f):
    def one(rows, cols):
        v, s = operands(rng, rows, cols, g)
        return v, (s * cols ** -0.5).astype(np.float32).astype(np.float64)
    return one(f, d), one(f, d), one(d, f)


@pytest.mark.parametrize("case", range(len(FFNS)))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_ffn(case, dtype):
    rows, d, f = FFNS[case]
    rng = np.random.default_rng(100 + case)
    offsets = np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)
    R = int(offsets[-1]) + 3
    x, xs = ref.quantize_tiles(rounded(rng.normal(size=(R, d)), "bf16"))
    W = ffn_weights(rng, len(rows), d, f)
    gate = rng.uniform(0.1, 1, size=R).astype(np.float32) if case % 2 else None
    out = run_ffn(codes_of(x), dev(xs), W, offsets, dtype, gate, R)
    got = host(out)
    assert (got[offsets[-1]:] == -7.0).all()
    for g in range(len(rows)):
        at = slice(offsets[g], offsets[g + 1])
        if rows[g] == 0:
            continue
        y, bound = ref.experts(x[at], xs[at], W[0][0][g], W[0][1][g], W[1][0][g], W[1][1][g], W[2][0][g], W[2][1][g])
        sc = 1.0 if gate is None else gate[at, None].astype(np.float64)
        close(got[at], y * sc, (bound + 2 * U32 * np.abs(y)) * sc + (half_step(dtype) + U32) * np.abs(y * sc))


# ---------------------------------------------------------------------------
# streams, graphs
# ---------------------------------------------------------------------------
def test_captured_and_replayed_with_new_inputs():
    """Norm, product and dropout captured together; replays read new inputs and draw new masks."""
    rng = np.random.default_rng(60)
    n, d, f = 70, 256, 320
    x = dev(rng.normal(size=(n, d)), torch.bfloat16)
    w, wsc = operands(rng, f, d, 1)
    wc, wsd = codes_of(w), dev(wsc)
    res = dev(rng.normal(size=(n, f)), torch.bfloat16)
    words = rng_words(1, 0)
    codes, scales = filled((n, d), torch.uint8, 0), filled((n, blocks(d)), torch.float32)
    y, out = filled((n, f), torch.bfloat16), filled((n, f), torch.bfloat16)
    ws = moe.alloc_workspace(moe.moe_block_matmul_workspace_size(1, f, d, n))

    def step():
        moe.moe_layer_norm(x, moe.DTYPE_BF16, n, d, moe.NORM_RMS, None, None, 1e-6, None, None, None, codes, scales)
        moe.moe_block_matmul(1, f, d, n, None, codes, scales, wc, wsd, None, moe.DTYPE_BF16, y, ws)
        moe.moe_dropout_add(y, res, moe.DTYPE_BF16, n * f, 0.3, words, out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.copy_(dev(rng.normal(size=(n, d)), torch.bfloat16))
        words[1] = 10 + i
        graph.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        out.fill_(-7.0)
        y.fill_(-7.0)
        step()
        torch.cuda.synchronize()
        assert torch.equal(out, replayed)
    assert moe.moe_get_device_error(ws) == 0


def test_calls_in_turn_share_a_workspace():
    """A workspace that the layer, a product cut into ranges, one that is not and the
    experts use in turn: the counters in its control block do not meet."""
    rng = np.random.default_rng(62)
    w = mi.WORKLOADS["deepseek_v3"].with_(T=64, d_model=256, E_r=16, E_s=0, K=2, d_ffn=128, n_groups=1, topk_groups=1,
                                          group_topn=0)
    cfg = moe.config_for(w)
    nbytes = max(moe.moe_workspace_size(cfg), moe.moe_block_matmul_workspace_size(1, 1500, 7168, 3),
                 moe.moe_block_matmul_workspace_size(1, 1500, 7168, 2000), moe.moe_block_ffn_workspace_size(1, 2048, 256, 2))
    ws = moe.alloc_workspace(nbytes)
    W = [dev(mi.gen_weight(w, k), torch.bfloat16) for k in ("gate", "up", "down")]
    h, e, y = dev(mi.gen_h(w), torch.bfloat16), dev(mi.gen_centroids(w)), filled((64, 256), torch.bfloat16)
    v, s = operands(rng, 2000, 7168)
    m, ms = operands(rng, 1500, 7168, 1)
    vc, sd, mc, msd = codes_of(v), dev(s), codes_of(m), dev(ms)
    few, many = filled((3, 1500), torch.float32), filled((2000, 1500), torch.float32)
    F = ffn_weights(rng, 1, 2048, 256)
    F = [(codes_of(a), dev(b)) for a, b in F]
    xq, xs = ref.quantize_tiles(rounded(rng.normal(size=(2, 2048)), "bf16"))
    xq, xs, out = codes_of(xq), dev(xs), filled((2, 2048), torch.float32)
    seen = []
    for _ in range(3):
        for t in (few, many, out, y):
            t.fill_(-7.0)
        moe.moe_layer_forward(cfg, h, e, None, *W, None, None, None, y, ws)
        moe.moe_block_matmul(1, 1500, 7168, 3, None, vc, sd, mc, msd, None, moe.DTYPE_F32, few, ws)
        moe.moe_block_matmul(1, 1500, 7168, 2000, None, vc, sd, mc, msd, None, moe.DTYPE_F32, many, ws)
        moe.moe_block_ffn(1, 2048, 256, 2, None, xq, xs, *F[0], *F[1], *F[2], None, moe.DTYPE_F32, out, ws)
        moe.moe_block_matmul(1, 1500, 7168, 3, None, vc, sd, mc, msd, None, moe.DTYPE_F32, few, ws)
        torch.cuda.synchronize()
        assert moe.moe_get_device_error(ws) == 0
        seen.append([t.clone() for t in (few, many, out, y)])
    for a, b in zip(seen[0] * 2, seen[1] + seen[2]):
        assert torch.equal(a, b)
    check_matmul(few, v[:3], s[:3], m, ms, [0, 3], "f32")
    check_matmul(many[:64], v[:64], s[:64], m, ms, [0, 64], "f32")


def test_on_a_stream_of_its_own():
    rng = np.random.default_rng(61)
    x, gamma, _, _ = norm_inputs(300, 512, "bf16", 9)
    t = dev(x, torch.bfloat16)
    want, _, _, _, _ = run_norm(t, "bf16", moe.NORM_RMS, dev(gamma), None)
    torch.cuda.synchronize()
    g = dev(gamma)
    side = torch.cuda.Stream()
    out = filled((300, 512), torch.bfloat16)
    torch.cuda.synchronize()
    moe.moe_layer_norm(t, moe.DTYPE_BF16, 300, 512, moe.NORM_RMS, g, None, 1e-6, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


# ---------------------------------------------------------------------------
# a run of them together
# ---------------------------------------------------------------------------
def small_layer():
    w = mi.WORKLOADS["deepseek_v3"].with_(T=200, d_model=256, E_r=32, E_s=1, K=4, d_ffn=128, d_ffn_shared=192,
                                          n_groups=4, topk_groups=2, group_topn=2)
    W = {k: mi.gen_weight(w, k) for k in ("gate", "up", "down", "sgate", "sup", "sdown")}
    cfg_o = mo.LayerConfig(T=w.T, d_model=w.d_model, E_r=w.E_r, E_s=w.E_s, K=w.K, n_groups=w.n_groups,
                           topk_groups=w.topk_groups, group_topn=w.group_topn)
    return w, W, cfg_o


def rms(a):
    return float(np.sqrt(np.mean(np.square(a))))


def test_serving_sublayer():
    """x + MoE(norm(x)) with block-scaled experts: the norm's e4m3 copy gathered into
    expert order, routed and shared experts, the combine with x as the residual."""
    w, W, cfg_o = small_layer()
    T, d, f, fs, E, K = w.T, w.d_model, w.d_ffn, w.d_ffn_shared, w.E_r, w.K
    rng = np.random.default_rng(70)
    x = rounded(rng.normal(size=(T, d)) * 3.0, "bf16")
    gamma = rng.uniform(0.5, 1.5, size=d).astype(np.float32)
    h64 = ref.norm(x, False, gamma)[0]
    s = mo.affinity(rounded(h64, "bf16"), mi.gen_centroids(w), 0)
    b = mi.gen_bias(w)
    Q = {k: ref.quantize_blocks(v) for k, v in W.items()}
    xq, xs = ref.quantize_tiles(rounded(h64, "bf16"))
    idx_o, gates_o, disp = mo.route(cfg_o, s, b)
    y64 = x.astype(np.float64)
    one = lambda rows, e, p, g: ref.experts(xq[rows], xs[rows], Q[p + "gate"][0][e], Q[p + "gate"][1][e], Q[p + "up"][0][e],  # noqa: E731
                                            Q[p + "up"][1][e], Q[p + "down"][0][e], Q[p + "down"][1][e])[0] * g
    y64 = y64 + one(np.arange(T), 0, "s", 1.0)
    for e in range(E):
        tok, slot = np.nonzero(idx_o == e)
        if tok.size:
            y64[tok] += one(tok, e, "", gates_o[tok, slot][:, None])

    cfg = moe.config_for(w)
    ws = moe.alloc_workspace(moe.moe_workspace_size(cfg))
    xd = dev(x, torch.bfloat16)
    codes, scales = filled((T, d), torch.uint8, 0), filled((T, blocks(d)), torch.float32)
    h = filled((T, d), torch.bfloat16)
    moe.moe_layer_norm(xd, moe.DTYPE_BF16, T, d, moe.NORM_RMS, dev(gamma), None, 1e-6, h, None, None, codes, scales)
    i32 = lambda *sh: filled(sh, torch.int32, -5)  # noqa: E731
    idx, gates, counts = i32(T, K), filled((T, K), torch.float32), i32(E)
    moe.moe_route(cfg, h, None, dev(b), dev(s), None, idx, gates, counts, ws)
    off, tok, row_of, kept, rg = i32(E + 1), i32(T * K), i32(T, K), i32(E), filled((T * K,), torch.float32)
    moe.moe_permute(cfg, idx, gates, None, off, tok, row_of, kept, rg, None, ws)
    cp, sp = filled((T * K, d), torch.uint8, 0), filled((T * K, blocks(d)), torch.float32)
    moe.moe_gather_rows(codes, T, d, tok, T * K, cp)
    moe.moe_gather_rows(scales, T, 4 * blocks(d), tok, T * K, sp)
    D = {}
    for k, v in W.items():
        n, r, c = v.shape
        D[k] = (filled((n, r, c), torch.uint8, 0), filled((n, blocks(r), blocks(c)), torch.float32))
        moe.moe_quantize_blocks(dev(v, torch.bfloat16), moe.DTYPE_BF16, n, r, c, *D[k])
    slot, shared, y = filled((T * K, d), torch.bfloat16), filled((1, T, d), torch.bfloat16), filled((T, d), torch.bfloat16)
    wf = moe.alloc_workspace(max(moe.moe_block_ffn_workspace_size(E, d, f, T * K),
                                 moe.moe_block_ffn_workspace_size(1, d, fs, T)))
    moe.moe_block_ffn(E, d, f, T * K, off, cp, sp, *D["gate"], *D["up"], *D["down"], rg, moe.DTYPE_BF16, slot, wf)
    moe.moe_block_ffn(1, d, fs, T, None, codes, scales, *D["sgate"], *D["sup"], *D["sdown"], None, moe.DTYPE_BF16,
                      shared, wf)
    moe.moe_combine(cfg, xd, slot, shared, row_of, y)
    assert np.array_equal(idx.cpu().numpy(), idx_o)
    assert moe.moe_get_device_error(wf) == 0 and moe.moe_get_device_error(ws) == 0
    # the layer's bar: each expert row is rounded to bf16 once before the sum, and
    # a bf16 rounding of the norm may fall on the other side
    assert np.max(np.abs(host(y) - y64)) <= 2e-2 * rms(y64)
    assert np.max(np.abs(host(y) - y64) - 2.0 ** -8 * np.abs(y64)) <= 2e-2 * rms(y64 - x)


def test_training_sublayer():
    """x + dropout(MoE(norm(x))) forward and backward around the layer's own pass."""
    w, W, cfg_o = small_layer()
    T, d, p, seed = w.T, w.d_model, 0.2, 99
    rng = np.random.default_rng(71)
    x = rounded(rng.normal(size=(T, d)) * 3.0 + 0.5, "bf16")
    gamma, beta = rng.uniform(0.5, 1.5, size=d).astype(np.float32), rng.normal(size=d).astype(np.float32)
    dy = rounded(rng.normal(size=(T, d)), "bf16")
    e, b = mi.gen_centroids(w), mi.gen_bias(w)
    n64, mean, rstd = ref.norm(x, True, gamma, beta)
    h = rounded(n64, "bf16")
    s = mo.affinity(h, e, 0)
    cfg_o.add_residual = 0
    source = lambda which, ex: W[which][ex]  # noqa: E731
    fwd = mo.layer_forward(cfg_o, h, e, b, source, s_in=s)
    keep = ref.keep_mask(seed, 5, T * d, p).reshape(T, d)
    y64 = x + np.where(keep, fwd["y"] / (1 - p), 0.0)
    dm64 = np.where(keep, dy / (1 - p), 0.0)
    idx_o, gates_o, disp_o = mo.route(cfg_o, s, b)
    bwd = mo.layer_backward(cfg_o, h, e, s, idx_o, gates_o, disp_o, source, dm64)
    dx64, dg64, db64, _ = ref.norm_backward(bwd["dh"], x, True, gamma, mean, rstd, dy)

    BF = torch.bfloat16
    cfg = moe.config_for(w, train=1, add_residual=0)
    ws = moe.alloc_workspace(moe.moe_workspace_size(cfg))
    xd, words, g, be = dev(x, BF), rng_words(seed, 5), dev(gamma), dev(beta)
    hd, m, y = filled((T, d), BF), filled((T, d), BF), filled((T, d), BF)
    mu, rs = filled((T,), torch.float32), filled((T,), torch.float32)
    idx = filled((T, w.K), torch.int32, -5)
    D = {k: dev(v, BF) for k, v in W.items()}
    names = ("gate", "up", "down", "sgate", "sup", "sdown")
    moe.moe_layer_norm(xd, moe.DTYPE_BF16, T, d, moe.NORM_LAYER, g, be, 1e-6, hd, mu, rs)
    moe.moe_layer_forward(cfg, hd, dev(e), dev(b), *[D[k] for k in names], m, ws, s_in=dev(s), idx_out=idx)
    moe.moe_dropout_add(m, xd, moe.DTYPE_BF16, T * d, p, words, y)
    dm, dh, dx = filled((T, d), BF), filled((T, d), BF), filled((T, d), BF)
    de, dg, db = filled((w.E_r, d), torch.float32), filled((d,), torch.float32), filled((d,), torch.float32)
    G = [torch.empty_like(D[k]) for k in names]
    wn = moe.alloc_workspace(moe.moe_layer_norm_backward_workspace_size(T, d))
    dyd = dev(dy, BF)
    moe.moe_dropout_backward(dyd, moe.DTYPE_BF16, T * d, p, words, dm)
    moe.moe_layer_backward(cfg, hd, dev(e), dev(s), idx, *[D[k] for k in names], dm, dh, de, *G, ws)
    moe.moe_layer_norm_backward(dh, xd, moe.DTYPE_BF16, T, d, moe.NORM_LAYER, g, mu, rs, dyd, dx, dg, db, wn)
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == 0
    assert np.array_equal(idx.cpu().numpy(), idx_o)
    # the layer's bars (2 % of the RMS forward, 3 % backward), the dropout's scale on top
    assert np.max(np.abs(host(y) - y64) - 2.0 ** -8 * np.abs(y64)) <= 2e-2 * rms(y64 - x) / (1 - p)
    for got, want in ((dx, dx64), (dg, dg64), (db, db64)):
        assert np.max(np.abs(host(got) - want) - 2.0 ** -8 * np.abs(want)) <= 3e-2 * rms(want) / (1 - p)
