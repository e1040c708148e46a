"""Performance cases of the operators around and inside a sparse expert sublayer
x + dropout(MoE(norm(x))):

* the layer norm in front of the router and its backward pass (with the reduction
  of the gain's and bias's gradients), on its own and with the e4m3 copy of its
  output that the block-scaled experts read;
* dropout with the residual behind the experts, its mask drawn from a counter and
  never stored, and its backward pass;
* grouped matrix products in e4m3 with one scale for each block of 128 (activations
  1 x 128, weights 128 x 128), and the SwiGLU experts made of them.

`run` computes an operator in plain torch operations, or with `own` through the
library's entry points.  `exact` computes the same from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
E4M3 = torch.float8_e4m3fn
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# the largest listed case's weights (one matrix) and multiply-adds (one product): drawn cases stay below
MOST_WEIGHTS, MOST_WORK, MOST_VALUES = 256 * 2048 * 7168, 32768 * 2048 * 7168, 4096 * 7168


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a decode step's 64 tokens: root-mean-square norm with the e4m3 copy for the experts
        {"name": "norm decode", "op": "norm", "rows": 64, "d": 7168, "dtype": "bf16", "kind": "rms", "tiles": True},
        # a prefill or training batch's norm
        {"name": "norm batch", "op": "norm", "rows": 4096, "d": 7168, "dtype": "bf16", "kind": "layer", "tiles": False},
        # odd rows and width in fp32: no row but the first is aligned to more than four bytes
        {"name": "norm odd fp32", "op": "norm", "rows": 511, "d": 1001, "dtype": "f32", "kind": "layer", "tiles": False},
        # a training step's backward of the norm, with the residual's gradient added
        {"name": "norm grad batch", "op": "norm_grad", "rows": 4096, "d": 7168, "dtype": "bf16", "kind": "layer", "residual": True},
        # the toy layer's norm backward: latency
        {"name": "norm grad toy", "op": "norm_grad", "rows": 512, "d": 64, "dtype": "f32", "kind": "rms", "residual": False},
        # a training batch's expert outputs dropped and added to the residual stream
        {"name": "dropout batch", "op": "dropout", "rows": 4096, "d": 7168, "dtype": "bf16", "p": 0.1},
        # the gradient behind a fine-grained layer, the mask drawn again; an odd number of rows
        {"name": "dropout grad fp32", "op": "dropout_grad", "rows": 8191, "d": 2048, "dtype": "f32", "p": 0.4},
        # one token through the shared expert's gate matrix
        {"name": "matmul one token", "op": "matmul", "experts": 1, "active": 1, "rows": 1, "n": 2048, "k": 7168, "gated": False, "dtype": "bf16"},
        # a fine-grained layer with ragged experts, some without rows, fewer columns than whole tiles hold
        {"name": "matmul ragged", "op": "matmul", "experts": 64, "active": 61, "rows": 4099, "n": 1400, "k": 2032, "gated": True, "dtype": "bf16"},
        # a batch over few wide experts: bound by the products
        {"name": "matmul wide", "op": "matmul", "experts": 8, "active": 8, "rows": 8192, "n": 14336, "k": 4096, "gated": False, "dtype": "bf16"},
        # a decode step of 64 tokens over fine-grained experts: bound by the weights of the experts that have rows
        {"name": "experts decode", "op": "experts", "experts": 256, "active": 150, "rows": 512, "d": 7168, "f": 2048, "dtype": "bf16"},
        # a batch of 4096 tokens over the same experts
        {"name": "experts batch", "op": "experts", "experts": 256, "active": 256, "rows": 32768, "d": 7168, "f": 2048, "dtype": "bf16"},
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "dropout", "dropout_grad", "matmul", "experts"])
    if op in ("norm", "norm_grad", "dropout", "dropout_grad"):
        d = spread(rng, 64, 8192)
        rows = spread(rng, 1, min(16384, MOST_VALUES // d))
        case = {"op": op, "rows": rows, "d": d, "dtype": rng.choice(["f32", "bf16"])}
        if op == "norm":
            case.update(kind=rng.choice(["layer", "rms"]), tiles=rng.random() < 0.4)
            if case["tiles"]:
                case["d"] = d // 16 * 16
        elif op == "norm_grad":
            case.update(kind=rng.choice(["layer", "rms"]), residual=rng.random() < 0.5)
        else:
            case.update(p=rng.choice([0.1, 0.25, 0.4]))
        return case
    experts = spread(rng, 1, 256)
    active = max(1, int(experts * rng.uniform(0.5, 1.0)))
    if op == "matmul":
        k = 16 * spread(rng, 8, 512)
        n = spread(rng, 64, max(64, min(14336, MOST_WEIGHTS // (experts * k))))
        case = {"op": op, "experts": experts, "active": active, "n": n, "k": k, "gated": rng.random() < 0.5, "dtype": "bf16"}
    else:
        k = 16 * spread(rng, 8, 448)
        n = 16 * spread(rng, 4, max(4, min(14336, MOST_WEIGHTS // (experts * k)) // 16))
        case = {"op": op, "experts": experts, "active": active, "d": k, "f": n, "dtype": "bf16"}
    rows = min(32768, MOST_WORK // (n * k), 200_000_000 // max(n, k))
    case["rows"] = spread(rng, active, max(active, rows))
    return case


def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "f32" else 2
    if op in ("norm", "norm_grad", "dropout", "dropout_grad"):
        r, d = case["rows"], case["d"]
        if op == "norm":
            moved = 2 * r * d * size + 8 * d + 8 * r + ((r * d + 4 * r * blocks(d)) if case["tiles"] else 0)
            return {"bytes": moved, "flops": 8 * r * d}
        if op == "norm_grad":
            return {"bytes": (3 + case["residual"]) * r * d * size + 12 * d + 8 * r, "flops": 14 * r * d}
        return {"bytes": (3 if op == "dropout" else 2) * r * d * size, "flops": 4 * r * d}
    a, r = case["active"], case["rows"]
    if op == "matmul":
        n, k = case["n"], case["k"]
        moved = a * (n * k + 4 * blocks(n) * blocks(k)) + r * (k + 4 * blocks(k)) + r * n * size + 4 * case["experts"]
        return {"bytes": moved, "flops": 2 * r * n * k}
    d, f = case["d"], case["f"]
    moved = 3 * a * (d * f + 4 * blocks(d) * blocks(f)) + 2 * r * d + r * d * size + 4 * case["experts"]
    return {"bytes": moved, "flops": 6 * r * d * f}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def rows_of_experts(case, seed):
    """Rows of each expert: `active` of them have at least one, unevenly."""
    rng = np.random.default_rng([seed, 7])
    live = rng.permutation(case["experts"])[: case["active"]]
    share = rng.lognormal(0.0, 0.5, size=live.size)
    n = np.zeros(case["experts"], np.int64)
    n[live] = 1 + rng.multinomial(case["rows"] - live.size, share / share.sum())
    return n


def e4m3_weights(g, dev, n_mats, rows, cols):
    """Codes of n_mats matrices whose blocks fill the type's range, and a scale for each block."""
    codes = torch.empty((n_mats, rows, cols), dtype=E4M3, device=dev)
    step = max(1, 500_000_000 // (rows * cols))
    for at in range(0, n_mats, step):
        part = codes[at:at + step]
        part.copy_(torch.randn(part.shape, generator=g, device=dev).mul_(106.0).clamp_(-448.0, 448.0))
    scales = torch.randn((n_mats, blocks(rows), blocks(cols)), generator=g, device=dev).mul_(0.3).exp_()
    return codes, scales.mul_(cols ** -0.5 / 106.0)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    randn = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    st = {"case": case}
    if op in ("norm", "norm_grad", "dropout", "dropout_grad"):
        r, d = case["rows"], case["d"]
        # a residual stream: channels of different size, a few of them large, an offset
        x = (randn(r, d) * randn(d).mul_(0.8).exp_() + 0.3 * randn(d)).to(dt)
        if op in ("norm", "norm_grad"):
            st.update(x=x, gamma=1.0 + 0.1 * randn(d), beta=0.1 * randn(d) if case["kind"] == "layer" else None, eps=1e-6)
            st["rstd"] = torch.empty(r, device=dev)
            st["mean"] = torch.empty(r, device=dev) if case["kind"] == "layer" else None
        if op == "norm":
            st["out"] = torch.empty_like(x)
            if case["tiles"]:
                st["codes"] = torch.empty((r, d), dtype=E4M3, device=dev)
                st["scales"] = torch.empty((r, blocks(d)), device=dev)
                st["values"] = torch.empty((r, blocks(d), BLOCK), dtype=torch.bfloat16, device=dev)
        elif op == "norm_grad":
            xf = x.double()
            mean = xf.mean(1) if case["kind"] == "layer" else torch.zeros(r, dtype=torch.float64, device=dev)
            st["rstd"].copy_(((xf - mean[:, None]).square().mean(1) + st["eps"]).rsqrt())
            if st["mean"] is not None:
                st["mean"].copy_(mean)
            st["dy"] = (0.02 * randn(r, d)).to(dt)
            st["dres"] = (0.02 * randn(r, d)).to(dt) if case["residual"] else None
            st.update(dx=torch.empty_like(x), dgamma=torch.empty(d, device=dev),
                      dbeta=torch.empty(d, device=dev) if case["kind"] == "layer" else None)
        else:
            st.update(x=x, res=randn(r, d).to(dt) if op == "dropout" else None, out=torch.empty_like(x))
            # the generator's seed, and the number of this draw
            st["rng"] = torch.randint(0, 2 ** 62, (2,), generator=g, device=dev, dtype=torch.int64)
        return st
    rows = rows_of_experts(case, seed)
    offsets = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    st.update(offsets=torch.from_numpy(offsets).to(dev), most=int(rows.max()))
    r = case["rows"]
    if op == "matmul":
        n, k = case["n"], case["k"]
        st["x"] = randn(r, k).mul_(130.0).clamp_(-448.0, 448.0).to(E4M3)
        st["x_scale"] = torch.exp2(randn(r, blocks(k)).round_() - 7.0)
        st["w"], st["w_scale"] = e4m3_weights(g, dev, case["experts"], n, k)
        st["out"] = torch.empty((r, n), dtype=dt, device=dev)
        st["gate"] = torch.rand(r, generator=g, device=dev).add_(0.05) if case["gated"] else None
    else:
        d, f = case["d"], case["f"]
        st["x"] = (randn(r, d) * randn(d).mul_(0.5).exp_()).to(torch.bfloat16)
        st["codes"] = torch.empty((r, d), dtype=E4M3, device=dev)
        st["scales"] = torch.empty((r, blocks(d)), device=dev)
        for name, a, b in (("gate", f, d), ("up", f, d), ("down", d, f)):
            st["w_" + name], st["s_" + name] = e4m3_weights(g, dev, case["experts"], a, b)
        st["gate"] = torch.rand(r, generator=g, device=dev).add_(0.05)
        st["out"] = torch.empty((r, d), dtype=dt, device=dev)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def spread_scales(scales, rows, cols):
    """The scale of every value of [.., rows, cols] from those of its 128 x 128 blocks."""
    return scales.repeat_interleave(BLOCK, -2)[..., :rows, :].repeat_interleave(BLOCK, -1)[..., :cols]


def tile_scales(v):
    """Scales of the 1 x 128 tiles of fp32 rows: the smallest power of two that brings a tile below 448."""
    r, c = v.shape
    padded = torch.zeros((r, blocks(c) * BLOCK), device=v.device)
    padded[:, :c] = v.abs()
    m, e = torch.frexp(padded.view(r, -1, BLOCK).amax(2))
    s = torch.ldexp(torch.ones_like(m), (e - 9 + (m > 0.875).int()).clamp(min=-126))
    return torch.where(m == 0, torch.ones_like(s), s)


def tile_values(v):
    """fp32 rows as their e4m3 codes and scales stand for them."""
    s = tile_scales(v).repeat_interleave(BLOCK, 1)[:, : v.shape[1]]
    return (v / s).to(E4M3).float() * s


def plain_norm(st):
    x = st["x"].float()
    mean = x.mean(1, keepdim=True) if st["mean"] is not None else 0.0
    c = x - mean
    rstd = (c.square().mean(1, keepdim=True) + st["eps"]).rsqrt()
    y = c * rstd * st["gamma"]
    if st["beta"] is not None:
        y = y + st["beta"]
    out = {"out": y.to(st["x"].dtype), "rstd": rstd[:, 0]}
    if st["mean"] is not None:
        out["mean"] = mean[:, 0]
    if st["case"]["tiles"]:
        out["tiles"] = tile_values(out["out"].float()).to(torch.bfloat16)
    return out


def plain_norm_grad(st):
    x, dy = st["x"].float(), st["dy"].float()
    rstd = st["rstd"][:, None]
    layer = st["mean"] is not None
    xhat = (x - st["mean"][:, None] if layer else x) * rstd
    gdy = dy * st["gamma"]
    dx = gdy - xhat * (gdy * xhat).mean(1, keepdim=True)
    if layer:
        dx = dx - gdy.mean(1, keepdim=True)
    dx = dx * rstd
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    out = {"dx": dx.to(st["x"].dtype), "dgamma": (dy * xhat).sum(0)}
    if layer:
        out["dbeta"] = dy.sum(0)
    return out


def times_32(a, b):
    """High and low 32 bits of a * b, a a tensor of 32-bit values in int64 and b a constant."""
    low, high = a * (b & 0xFFFF), a * (b >> 16)
    mid = high + (low >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (low & 0xFFFF)


def plain_uniform(rng, n):
    """n values in [0, 1): 32-bit words of Philox4x32-10 (Salmon et al., 2011), key the
    seed, counter (i / 4, number of the draw), word i % 4 for value i."""
    q = torch.arange((n + 3) // 4, device=rng.device)
    part = lambda v, at: (v >> at) & 0xFFFFFFFF  # noqa: E731
    c0, c1 = part(q, 0), part(q, 32)
    c2, c3 = part(rng[1], 0) + 0 * q, part(rng[1], 32) + 0 * q
    k0, k1 = part(rng[0], 0), part(rng[0], 32)
    for _ in range(10):
        (h0, l0), (h1, l1) = times_32(c0, 0xD2511F53), times_32(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return torch.stack([c0, c1, c2, c3], 1).view(-1)[:n].double() / 2.0 ** 32


def plain_dropout(st):
    x, p = st["x"].float(), st["case"]["p"]
    keep = plain_uniform(st["rng"], x.numel()).view(x.shape) >= p
    y = torch.where(keep, x * (1.0 / (1.0 - p)), torch.zeros_like(x))
    if st["res"] is not None:
        y = y + st["res"].float()
    return y.to(st["x"].dtype)


def by_expert(st, rows):
    """Rows in expert order as [experts, most, cols], padded with zeros, and where each row went."""
    off = st["offsets"].long()
    at = torch.arange(rows.shape[0], device=rows.device)
    e = torch.searchsorted(off, at, right=True) - 1
    place = e * st["most"] + at - off[e]
    padded = torch.zeros((st["case"]["experts"] * st["most"], rows.shape[1]), device=rows.device)
    padded[place] = rows
    return padded.view(st["case"]["experts"], st["most"], -1), place


def plain_product(st, rows, w, s):
    padded, place = by_expert(st, rows)
    wf = w.float().mul_(spread_scales(s, w.shape[1], w.shape[2]))
    return torch.bmm(padded, wf.transpose(1, 2)).view(-1, w.shape[1])[place]


def plain_matmul(st):
    x = st["x"].float()
    x *= st["x_scale"].repeat_interleave(BLOCK, 1)[:, : x.shape[1]]
    y = plain_product(st, x, st["w"], st["w_scale"])
    if st["gate"] is not None:
        y = y * st["gate"][:, None]
    return y.to(st["out"].dtype)


def plain_experts(st):
    x = tile_values(st["x"].float())
    u = plain_product(st, x, st["w_gate"], st["s_gate"])
    v = plain_product(st, x, st["w_up"], st["s_up"])
    a = tile_values(u / (1.0 + torch.exp(-u)) * v)
    y = plain_product(st, a, st["w_down"], st["s_down"])
    return (y * st["gate"][:, None]).to(st["out"].dtype)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def library_workspace(st, nbytes):
    """The workspace that a program keeps for its calls."""
    import sparse_mixture_experts_selection_b200 as moe
    if "ws" not in st:
        st["ws"] = moe.alloc_workspace(nbytes())
    return st["ws"]


def library_run(st):
    import sparse_mixture_experts_selection_b200 as moe
    case = st["case"]
    op, r = case["op"], case["rows"]
    dt = moe.DTYPE_F32 if case["dtype"] == "f32" else moe.DTYPE_BF16
    if op in ("norm", "norm_grad"):
        kind = moe.NORM_LAYER if case["kind"] == "layer" else moe.NORM_RMS
    if op == "norm":
        moe.moe_layer_norm(st["x"], dt, r, case["d"], kind, st["gamma"], st["beta"], st["eps"], st["out"],
                           st["mean"], st["rstd"], st.get("codes"), st.get("scales"))
        out = {"out": st["out"], "rstd": st["rstd"]}
        if st["mean"] is not None:
            out["mean"] = st["mean"]
        if case["tiles"]:
            # the codes as the values they stand for: exact in bf16
            v = st["codes"].to(torch.bfloat16)
            if case["d"] % BLOCK == 0:
                out["tiles"] = torch.mul(v.view(r, -1, BLOCK), st["scales"][:, :, None], out=st["values"]).view(r, -1)
            else:
                out["tiles"] = v * st["scales"].to(torch.bfloat16).repeat_interleave(BLOCK, 1)[:, : case["d"]]
        return out
    if op == "norm_grad":
        ws = library_workspace(st, lambda: moe.moe_layer_norm_backward_workspace_size(r, case["d"]))
        moe.moe_layer_norm_backward(st["dy"], st["x"], dt, r, case["d"], kind, st["gamma"], st["mean"], st["rstd"],
                                    st["dres"], st["dx"], st["dgamma"], st["dbeta"], ws)
        out = {"dx": st["dx"], "dgamma": st["dgamma"]}
        if st["dbeta"] is not None:
            out["dbeta"] = st["dbeta"]
        return out
    if op == "dropout":
        moe.moe_dropout_add(st["x"], st["res"], dt, st["x"].numel(), case["p"], st["rng"], st["out"])
        return st["out"]
    if op == "dropout_grad":
        moe.moe_dropout_backward(st["x"], dt, st["x"].numel(), case["p"], st["rng"], st["out"])
        return st["out"]
    g = case["experts"]
    if op == "matmul":
        ws = library_workspace(st, lambda: moe.moe_block_matmul_workspace_size(g, case["n"], case["k"], r))
        moe.moe_block_matmul(g, case["n"], case["k"], r, st["offsets"], st["x"], st["x_scale"], st["w"],
                             st["w_scale"], st["gate"], dt, st["out"], ws)
        return st["out"]
    d, f = case["d"], case["f"]
    ws = library_workspace(st, lambda: moe.moe_block_ffn_workspace_size(g, d, f, r))
    moe.moe_quantize_tiles(st["x"], moe.DTYPE_BF16, r, d, st["codes"], st["scales"])
    moe.moe_block_ffn(g, d, f, r, st["offsets"], st["codes"], st["scales"], st["w_gate"], st["s_gate"], st["w_up"],
                      st["s_up"], st["w_down"], st["s_down"], st["gate"], dt, st["out"], ws)
    return st["out"]


PLAIN = {"norm": plain_norm, "norm_grad": plain_norm_grad, "dropout": plain_dropout, "dropout_grad": plain_dropout,
         "matmul": plain_matmul, "experts": plain_experts}


def run(state):
    if own:
        return library_run(state)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact_keep(seed, number, n, p):
    """The dropout mask from 64-bit whole numbers on the host."""
    q = np.arange((n + 3) // 4, dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    c = [q & low, q >> np.uint64(32), np.full_like(q, number & 0xFFFFFFFF), np.full_like(q, number >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1).reshape(-1)[:n] >= np.uint64(math.ceil(p * 2.0 ** 32))


def exact_tiles(v):
    """Rows through 1 x 128 tiles of e4m3 with power-of-two scales, in 64 bits: the codes' grid
    has steps of 2^(e - 3) in [2^e, 2^(e + 1)), at least 2^-9; ties go to the even code."""
    out = torch.empty_like(v)
    for at in range(0, v.shape[1], BLOCK):
        t = v[:, at:at + BLOCK]
        top = t.abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(top > 0, top, 448.0) / 448.0))
        e = torch.where(torch.exp2(e - 1) * 448.0 >= top, e - 1, e)
        e = torch.where(torch.exp2(e) * 448.0 < top, e + 1, e).clamp(min=-126)
        s = torch.where(top > 0, torch.exp2(e), 1.0)
        step = torch.exp2(torch.frexp(t / s)[1].double().sub(4).clamp(min=-9))
        out[:, at:at + BLOCK] = torch.round(t / s / step) * step * s
    return out


def exact_weight(w, s, e):
    m = w[e].double()
    rows = torch.arange(m.shape[0], device=m.device) // BLOCK
    cols = torch.arange(m.shape[1], device=m.device) // BLOCK
    return m * s[e].double()[rows][:, cols]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = st["x"].double()
        if case["kind"] == "layer":
            var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        else:
            var, mean = torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / case["d"], torch.zeros_like(x[:, :1])
        scale = 1.0 / torch.sqrt(var + st["eps"])
        out = {"out": (x - mean) * scale * st["gamma"].double() + (0.0 if st["beta"] is None else st["beta"].double()),
               "rstd": scale[:, 0]}
        if case["kind"] == "layer":
            out["mean"] = mean[:, 0]
        if case["tiles"]:
            out["tiles"] = exact_tiles(out["out"].to(DTYPES[case["dtype"]]).double())
        return out
    if op == "norm_grad":
        # the derivative of sum(dy * norm(x)) in 64 bits
        x, gamma, beta = (v.double().requires_grad_() for v in (st["x"], st["gamma"], torch.zeros_like(st["gamma"])))
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        if case["kind"] == "rms":
            var, mean = (x * x).mean(1, keepdim=True), 0.0
        y = (x - mean) / torch.sqrt(var + st["eps"]) * gamma + beta
        dx, dgamma, dbeta = torch.autograd.grad(y, (x, gamma, beta), st["dy"].double())
        out = {"dx": dx if st["dres"] is None else dx + st["dres"].double(), "dgamma": dgamma}
        if case["kind"] == "layer":
            out["dbeta"] = dbeta
        return out
    if op in ("dropout", "dropout_grad"):
        seed_, number = (int(v) for v in st["rng"].tolist())
        keep = torch.from_numpy(exact_keep(seed_, number, st["x"].numel(), case["p"])).to(st["x"].device)
        y = st["x"].double() * keep.view(st["x"].shape) / (1.0 - case["p"])
        return y + st["res"].double() if st["res"] is not None else y
    ends = st["offsets"].tolist()
    y = torch.zeros(st["out"].shape, dtype=torch.float64, device=st["out"].device)
    x = exact_tiles(st["x"].double()) if op == "experts" else None
    for e in range(case["experts"]):
        at = slice(ends[e], ends[e + 1])
        if ends[e] == ends[e + 1]:
            continue
        if op == "matmul":
            cols = torch.arange(case["k"], device=y.device) // BLOCK
            y[at] = (st["x"][at].double() * st["x_scale"][at].double()[:, cols]) @ exact_weight(st["w"], st["w_scale"], e).T
        else:
            u = x[at] @ exact_weight(st["w_gate"], st["s_gate"], e).T
            a = u * torch.sigmoid(u) * (x[at] @ exact_weight(st["w_up"], st["s_up"], e).T)
            y[at] = exact_tiles(a) @ exact_weight(st["w_down"], st["s_down"], e).T
    return y * st["gate"].double()[:, None] if st["gate"] is not None else y
