"""The operators around and inside the expert sublayer without a GPU: the plain
references against what fixes them, and every refusal of the entry points (each
call below fails its checks before any CUDA call)."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_mixture_experts_selection_b200 as moe
from oracle import moe_oracle as mo
import sublayer_reference as ref

P = 1 << 20            # an aligned, never-dereferenced stand-in for a device pointer
BF, F32 = moe.DTYPE_BF16, moe.DTYPE_F32


def test_philox_known_answers():
    """The published known-answer words of Philox4x32-10 for a zero counter and key."""
    got = ref.philox(np.zeros((1, 4), np.uint64), (0, 0))[0]
    assert [f"{int(v):08x}" for v in got] == ["6627e8d5", "e169c58d", "bc57ac4c", "9b00dbd8"]


def test_keep_mask_counts_and_addresses():
    keep = ref.keep_mask(5, 9, 1 << 20, 0.25)
    # a binomial with standard deviation 443: six of them
    assert abs(int(keep.sum()) - 3 * (1 << 18)) < 6 * 443.5
    assert np.array_equal(ref.keep_mask(5, 9, 100, 0.25, first=400), keep[400:500])
    assert not np.array_equal(ref.keep_mask(5, 10, 4096, 0.25), keep[:4096])
    assert ref.keep_mask(1, 2, 64, 0.0).all() and not ref.keep_mask(1, 2, 64, 1.0).any()


def test_grid_is_e4m3_and_tiles_follow_the_row_rule():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(codes.double().numpy(), ref.E4M3)
    rng = np.random.default_rng(0)
    v = rng.normal(size=4000) * np.exp2(rng.integers(-12, 8, size=4000))
    v = np.clip(v.astype(np.float32), -448, 448)
    assert np.array_equal(ref.to_grid(v), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())
    x = (rng.normal(size=(9, 128)) * np.exp2(rng.integers(-30, 30, size=(9, 1)))).astype(np.float32)
    q, s = ref.quantize_tiles(x)
    want_c, want_s = mo.quantize_rows(x)                # one tile is one row
    assert np.array_equal(ref.encode(q), want_c) and np.array_equal(s[:, 0], want_s.astype(np.float64))


@pytest.mark.parametrize("layer", [True, False])
def test_norm_backward_reference_against_differences(layer):
    rng = np.random.default_rng(3)
    x, dy, gamma, beta = rng.normal(size=(3, 11)), rng.normal(size=(3, 11)), rng.normal(size=11), rng.normal(size=11)
    loss = lambda x, g, b: float((ref.norm(x, layer, g, b)[0] * dy).sum())  # noqa: E731
    _, mean, rstd = ref.norm(x, layer, gamma, beta)
    dx, dg, db, _ = ref.norm_backward(dy, x, layer, gamma, mean, rstd)
    h = 1e-5
    for got, at in ((dx, 0), (dg, 1), (db, 2)):
        args = [x, gamma, beta]
        for i in np.ndindex(got.shape):
            v = []
            for sign in (1, -1):
                moved = [a.copy() for a in args]
                moved[at][i] += sign * h
                v.append(loss(*moved))
            # differences: h^2 times a third derivative, and rounding 1e-16 / h
            assert abs((v[0] - v[1]) / (2 * h) - got[i]) < 1e-7 * (1 + abs(got[i]))


def status(fn, *args):
    return getattr(moe.lib(), fn)(*args)


@pytest.mark.parametrize("change,want", [
    (dict(dtype=2), 1), (dict(n=-1), 1), (dict(n=1 << 40), 2), (dict(d=0), 1), (dict(d=16385), 2), (dict(kind=2), 1),
    (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(x=None), 1), (dict(x=P + 8), 1), (dict(out=None), 1), (dict(out=P + 2), 1), (dict(gamma=P + 2), 1),
    (dict(codes=P), 1), (dict(scales=P), 1), (dict(codes=P, scales=P, d=24), 1), (dict(codes=P + 4, scales=P), 1),
    (dict(rstd=P + 1), 1),
])
def test_norm_refusals(change, want):
    a = dict(x=P, dtype=BF, n=4, d=64, kind=0, gamma=P, beta=P, eps=1e-5, out=P, mean=P, rstd=P, codes=None, scales=None)
    a.update(change)
    assert status("moe_layer_norm", *a.values(), None) == want, moe.lib().moe_last_error_detail()


@pytest.mark.parametrize("change,want", [
    (dict(dtype=7), 1), (dict(n=-2), 1), (dict(d=20000), 2), (dict(kind=-1), 1), (dict(dy=None), 1), (dict(x=P + 4), 1),
    (dict(mean=None), 1), (dict(rstd=None), 1), (dict(dres=P + 2), 1), (dict(dx=None), 1), (dict(dgamma=P + 2), 1),
    (dict(ws=None), 3), (dict(ws=P + 16), 3), (dict(bytes=255), 3),
])
def test_norm_backward_refusals(change, want):
    need = moe.moe_layer_norm_backward_workspace_size(4, 64)
    a = dict(dy=P, x=P, dtype=BF, n=4, d=64, kind=0, gamma=P, mean=P, rstd=P, dres=P, dx=P, dgamma=P, dbeta=P, ws=P,
             bytes=need)
    a.update(change)
    assert status("moe_layer_norm_backward", *a.values(), None) == want, moe.lib().moe_last_error_detail()
    assert status("moe_layer_norm_backward_workspace_size", 4, 64, None) == 1


@pytest.mark.parametrize("change,want", [
    (dict(dtype=2), 1), (dict(n=-1), 1), (dict(p=-0.1), 1), (dict(p=1.01), 1), (dict(p=float("nan")), 1),
    (dict(x=None), 1), (dict(x=P + 2), 1), (dict(res=P + 2), 1), (dict(rng=None), 1), (dict(rng=P + 4), 1),
    (dict(out=None), 1), (dict(n=0, x=None, out=None, rng=None), 0),
])
def test_dropout_refusals(change, want):
    a = dict(x=P, res=P, dtype=BF, n=100, p=0.1, rng=P, out=P)
    a.update(change)
    assert status("moe_dropout_add", *a.values(), None) == want, moe.lib().moe_last_error_detail()
    if "res" not in change:
        a.pop("res")
        assert status("moe_dropout_backward", *a.values(), None) == want


def test_quantizer_refusals():
    for n, cols, dtype, src, codes, scales, want in (
            (4, 24, BF, P, P, P, 1), (4, 0, BF, P, P, P, 1), (-1, 32, BF, P, P, P, 1), (4, 32, 2, P, P, P, 1),
            (4, 32, BF, None, P, P, 1), (4, 32, BF, P + 8, P, P, 1), (4, 32, F32, P, P + 1, P, 1),
            (4, 32, F32, P, P, P + 2, 1), (4, (1 << 30) + 16, BF, P, P, P, 2), (0, 32, BF, None, None, None, 0)):
        assert status("moe_quantize_tiles", src, dtype, n, cols, codes, scales, None) == want
        assert status("moe_quantize_blocks", src, dtype, 1, n, cols, codes, scales, None) == want
    assert status("moe_quantize_blocks", P, BF, -1, 4, 32, P, P, None) == 1
    assert status("moe_quantize_blocks", P, BF, 1, (1 << 30) + 1, 32, P, P, None) == 2


@pytest.mark.parametrize("change,want", [
    (dict(g=0), 1), (dict(g=1025), 2), (dict(n=0), 1), (dict(k=8), 1), (dict(k=24), 1), (dict(rows=-1), 1),
    (dict(n=(1 << 20) + 1), 2), (dict(k=(1 << 20) + 16), 2), (dict(offsets=None), 1), (dict(offsets=P + 2), 1),
    (dict(x=None), 1), (dict(x=P + 8), 1), (dict(xs=None), 1), (dict(w=None), 1), (dict(w=P + 4), 1),
    (dict(wsc=P + 2), 1), (dict(scale=P + 2), 1), (dict(dtype=2), 1), (dict(out=None), 1), (dict(out=P + 8), 1),
    (dict(ws=None), 3), (dict(ws=P + 128), 3), (dict(bytes=16), 3), (dict(rows=0, x=None, out=None), 0),
])
def test_block_matmul_refusals(change, want):
    need = moe.moe_block_matmul_workspace_size(4, 100, 256, 50)
    a = dict(g=4, n=100, k=256, rows=50, offsets=P, x=P, xs=P, w=P, wsc=P, scale=P, dtype=BF, out=P, ws=P, bytes=need)
    a.update(change)
    assert status("moe_block_matmul", *a.values(), None) == want, moe.lib().moe_last_error_detail()
    n = ctypes.c_size_t(0)
    assert status("moe_block_matmul_workspace_size", 4, 100, 256, 50, None) == 1
    assert status("moe_block_matmul_workspace_size", 4, 100, 200, 50, ctypes.byref(n)) == 1


@pytest.mark.parametrize("change,want", [
    (dict(g=0), 1), (dict(g=2000), 2), (dict(d=24), 1), (dict(f=8), 1), (dict(rows=-1), 1), (dict(offsets=None), 1),
    (dict(x=P + 8), 1), (dict(xs=None), 1), (dict(wg=None), 1), (dict(sg=None), 1), (dict(wu=P + 4), 1),
    (dict(su=P + 2), 1), (dict(wd=None), 1), (dict(sd=None), 1), (dict(dtype=3), 1), (dict(out=None), 1),
    (dict(ws=None), 3), (dict(bytes=1000), 3), (dict(rows=0, x=None, out=None), 0),
])
def test_block_ffn_refusals(change, want):
    need = moe.moe_block_ffn_workspace_size(4, 128, 96, 50)
    a = dict(g=4, d=128, f=96, rows=50, offsets=P, x=P, xs=P, wg=P, sg=P, wu=P, su=P, wd=P, sd=P, scale=None,
             dtype=BF, out=P, ws=P, bytes=need)
    a.update(change)
    assert status("moe_block_ffn", *a.values(), None) == want, moe.lib().moe_last_error_detail()


def test_binding_refuses_tensors_the_kernels_cannot_take():
    """A strided view, another type, too few values or a host tensor never reach a launch."""
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    r = torch.zeros(8)
    for bad, word in ((torch.zeros(64, 8, dtype=torch.bfloat16).t(), "contiguous"), (x.float(), "type"),
                      (x[:4], "values"), (x, "GPU")):
        with pytest.raises(moe.MoeError, match=word):
            moe.moe_layer_norm(bad, BF, 8, 64, moe.NORM_RMS, None, None, 1e-6, x, None, r, stream=0)
    with pytest.raises(moe.MoeError, match="type"):
        moe.moe_dropout_add(x, None, BF, 8, 0.5, torch.zeros(2, dtype=torch.int32), x, stream=0)
    with pytest.raises(moe.MoeError, match="values"):
        moe.moe_block_matmul(3, 16, 64, 8, torch.zeros(3, dtype=torch.int32), x, r, x, r, None, BF, x, r, stream=0)


@pytest.mark.parametrize("rows,want", [((1 << 31) - 256, 0), ((1 << 31) - 255, 2), ((1 << 31) - 1, 2)])
def test_block_products_refuse_rows_that_whole_tiles_carry_past_32_bits(rows, want):
    """One group of so many rows: rounded up to tiles of 256 rows it must still be counted in 32 bits."""
    n = ctypes.c_size_t(0)
    assert status("moe_block_matmul_workspace_size", 1, 16, 16, rows, ctypes.byref(n)) == want
    assert status("moe_block_ffn_workspace_size", 1, 16, 16, rows, ctypes.byref(n)) == want
    if want:
        assert status("moe_block_matmul", 1, 16, 16, rows, None, P, P, P, P, None, BF, P, P, 1 << 40, None) == want
        assert status("moe_block_ffn", 1, 16, 16, rows, None, *[P] * 8, None, BF, P, P, 1 << 40, None) == want
        assert b"max_rows" in moe.lib().moe_last_error_detail()


def test_quantizers_refuse_sizes_whose_blocks_pass_64_bits():
    """No memory holds these, but a count of blocks that wraps round looks small."""
    top = 1 << 30
    for n_mats, rows, cols in ((1 << 18, top, top), ((1 << 31) - 1, top, top), (1 << 11, 1 << 17, 1 << 17)):
        assert status("moe_quantize_blocks", P, BF, n_mats, rows, cols, P, P, None) == 2
    for n_rows, cols in (((1 << 32) + 1, 16), (1 << 58, 16), (1 << 62, top)):
        assert status("moe_quantize_tiles", P, BF, n_rows, cols, P, P, None) == 2


@pytest.mark.parametrize("ws", [None, P])
def test_binding_needs_the_size_of_a_workspace(ws):
    """Plain addresses pass for arrays; a workspace without a size (none at all, or an
    address alone) is refused as the library refuses one that is too small."""
    calls = (lambda: moe.moe_layer_norm_backward(P, P, BF, 4, 64, 0, None, P, P, None, P, P, P, ws, stream=0),
             lambda: moe.moe_block_matmul(1, 16, 64, 4, None, P, P, P, P, None, BF, P, ws, stream=0),
             lambda: moe.moe_block_ffn(1, 64, 32, 4, None, *[P] * 8, None, BF, P, ws, stream=0))
    for call in calls:
        with pytest.raises(moe.MoeError, match="ws is") as e:
            call()
        assert e.value.status == 3


# the generator's other two published known answers: counter, key, words
PHILOX_ANSWERS = [
    ("ffffffff ffffffff ffffffff ffffffff", "ffffffff ffffffff", "408f276d 41c83b0e a20bc7c6 6d5451fd"),
    ("243f6a88 85a308d3 13198a2e 03707344", "a4093822 299f31d0", "d16cfe09 94fdcceb 5001e420 24126ea1"),
]


@pytest.mark.parametrize("counter,key,words", PHILOX_ANSWERS)
def test_philox_published_words_and_their_order(counter, key, words):
    """The published answers, and through them the order in which the seed, the number of the
    draw and a value's place fill the key and the counter: low words first."""
    c, k, w = ([int(v, 16) for v in t.split()] for t in (counter, key, words))
    assert ref.philox(np.array([c], np.uint64), k)[0].tolist() == w
    seed, draw, block = k[0] | k[1] << 32, c[2] | c[3] << 32, c[0] | c[1] << 32
    for p in (0.25, 0.5, 0.9):
        want = [v / 2.0 ** 32 >= p for v in w]
        assert ref.keep_mask(seed, draw, 4, p, first=4 * block).tolist() == want
    # words above and below each of them, one after the other
    for i in range(4):
        assert ref.keep_mask(seed, draw, 4, w[i] / 2.0 ** 32, first=4 * block)[i]
        assert not ref.keep_mask(seed, draw, 4, (w[i] + 1) / 2.0 ** 32, first=4 * block)[i]
