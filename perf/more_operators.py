"""Timed cases of the label head's residual features and 8-bit scores, and of gradient clipping.

    clip    norm = sqrt(sum over all tensors of g^2); out = min(1, max_norm / (norm + 1e-6)) g
    norm    h = x + residual, y = h rstd weight with rstd = (mean_j h^2 + eps)^-1/2;
            dx (of x and of the residual alike) and dweight from dy and the gradient of h
    norm8   the same forward, y in 8 bits: per row and block of 128 columns a power of two
            2^e, the least with max |y| <= 448 2^e, and q = y / 2^e in e4m3
    quant   rows in that form
    scores  out[i, v] = sum over blocks b of 2^(ea[i, b] + ew[v, b]) sum_{k in b} a[i, k] w[v, k]

Rows in 8 bits have their columns padded with zeros to whole blocks, and a row's
scales with ones to whole fours. With ``own`` false, ``run`` is the plain form:
elementary torch operations in float32 (the norm over all gradients in float64),
rounded once at the end. With ``own`` true it makes the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
Q8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6
MAX8 = 448.0  # the largest e4m3 value
BLOCK = 128


# ------------------------------------------------------------------ cases

def _clip(tensors, most, total, dtype, ratio):
    """tensors: how many, of 1 to `most` values each, about `total` in all; ratio: max_norm over the expected norm."""
    return dict(op="clip", tensors=tensors, most=most, total=total, dtype=dtype, ratio=ratio)


def _norm(n, dim, dtype, residual=True, affine=True, pad=0):
    return dict(op="norm", n=n, dim=dim, dtype=dtype, residual=residual, affine=affine, pad=pad)


def _norm8(n, dim, dtype, residual=True, affine=True, pad=0):
    return dict(op="norm8", n=n, dim=dim, dtype=dtype, residual=residual, affine=affine, pad=pad)


def _quant(n, dim, dtype, pad=0):
    return dict(op="quant", n=n, dim=dim, dtype=dtype, pad=pad)


def _scores(n, dim, vocab, dtype):
    return dict(op="scores", n=n, dim=dim, vocab=vocab, dtype=dtype)


def listed():
    return [
        # the four parameters of a small label head: launch latency is all there is
        dict(_clip(4, 110_592, 113_280, "f32", 0.5), name="clip_head"),
        # the five parameter arrays of a million-Gaussian scene
        dict(_clip(5, 48_000_000, 59_000_000, "f32", 0.5), name="clip_scene"),
        # many tensors of all sizes, odd ones among them, within the bound
        dict(_clip(300, 4_000_000, 40_000_000, "bf16", 2.0), name="clip_many"),
        # two codebook stages of every Gaussian of a million-Gaussian scene, a training step
        dict(_norm(1_000_000, 64, "f32"), name="norm_scene"),
        # wide features of odd row length in the columns of a wider matrix, a training step
        dict(_norm(32_771, 771, "bf16", pad=6), name="norm_odd"),
        # one picked Gaussian's features: latency
        dict(_norm8(1, 1024, "bf16"), name="norm8_pick"),
        # wide features of a batch of pixels, to be scored
        dict(_norm8(65_536, 1024, "bf16"), name="norm8_wide"),
        # a vocabulary of label texts, put into 8 bits once
        dict(_quant(65_536, 1024, "bf16"), name="quant_vocab"),
        # a float32 vocabulary of odd sizes
        dict(_quant(8_191, 129, "f32", pad=3), name="quant_odd"),
        # one picked Gaussian against an open vocabulary: the vocabulary is read once
        dict(_scores(1, 1024, 65_536, "f32"), name="scores_pick"),
        # a region's Gaussians, odd sizes
        dict(_scores(5_003, 129, 8_191, "f32"), name="scores_odd"),
        # a batch of pixels against an open vocabulary: the largest product
        dict(_scores(8_192, 1024, 65_536, "bf16"), name="scores_vocab"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _size(rng, lo, hi):
    """A size over the logarithm of the range: as drawn, or the next multiple of 64 if that is in it."""
    v = _log_uniform(rng, lo, hi)
    if rng.random() < 0.4:
        up = (v + 63) // 64 * 64
        v = up if up <= hi else v
    return v


def draw(rng):
    op = rng.choice(["clip", "norm", "norm8", "quant", "scores"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "clip":
        total = _log_uniform(rng, 1, 59_000_000)
        tensors = min(total, _log_uniform(rng, 1, 400))
        return _clip(tensors, max(1, _log_uniform(rng, (total + tensors - 1) // tensors, total)), total,
                     rng.choice(["f32", "bf16", "both"]), rng.choice([0.1, 0.5, 2.0]))
    if op in ("norm", "norm8", "quant"):
        n, dim = _size(rng, 1, 1_000_000), _size(rng, 1, 8192)
        n, pad = max(1, min(n, 64_000_000 // dim)), rng.choice([0, 0, 3, 8])
        if op == "quant":
            return _quant(n, dim, dtype, pad)
        make = _norm if op == "norm" else _norm8
        return make(n, dim, dtype, residual=rng.random() < 0.7, affine=rng.random() < 0.8, pad=pad)
    n, dim, vocab = _size(rng, 1, 65_536), _size(rng, 8, 8192), _size(rng, 2, 131_072)
    # at most the largest listed product, and its output's bytes
    vocab = max(2, min(vocab, 8_192 * 1024 * 65_536 // (n * dim), (1 << (29 if dtype == "bf16" else 28)) // n))
    return _scores(n, dim, vocab, dtype)


# ------------------------------------------------------------------ inputs

def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1_000_003 + salt)
    return g


def _randn(g, shape, dtype, pad=0):
    """Normal values; with ``pad`` the first columns of a matrix that much wider."""
    n, d = shape
    t = torch.randn((n, d + pad), generator=g, device=DEV, dtype=torch.float32).to(dtype)
    return t[:, :d]


def _sizes(case):
    """The tensors' sizes: the largest first, the others by a falling power, none empty, `total` in all but for
    what `most` cuts off."""
    k, most, left = case["tensors"], case["most"], case["total"]
    sizes = []
    for i in range(k):
        rest = k - 1 - i
        want = left - rest if rest == 0 else int(left * (0.83 if k < 10 else 0.05))
        sizes.append(max(1, min(most, want, left - rest)))
        left -= sizes[-1]
    return sizes


def _spread(g, dim):
    """Columns' spreads, as learned features have."""
    return torch.exp(0.5 * torch.randn(dim, generator=g, device=DEV))


def _padded(dim):
    """Columns of a row in 8 bits, and its scales."""
    cols = (dim + BLOCK - 1) // BLOCK * BLOCK
    return cols, (cols // BLOCK + 3) // 4 * 4


def prepare(case, seed):
    g = _gen(seed, 29)
    s = dict(case=case)
    if case["op"] == "clip":
        sizes = _sizes(case)
        kinds = [torch.float32, torch.bfloat16] if case["dtype"] == "both" else [TYPES[case["dtype"]]]
        kinds = [kinds[i % len(kinds)] for i in range(len(sizes))]
        # gradients of a factor of a hundred between tensors, as groups of parameters have
        size_of = [10.0 ** (i % 3 - 2) for i in range(len(sizes))]
        s["grads"] = [(torch.randn(k, generator=g, device=DEV) * a).to(t) for k, a, t in zip(sizes, size_of, kinds)]
        s["max_norm"] = case["ratio"] * math.sqrt(sum(k * a * a for k, a in zip(sizes, size_of)))
        # the clipped gradients go into flat buffers, one to a type
        s["flat"] = [torch.empty(sum(k for k, t in zip(sizes, kinds) if t is kind), dtype=kind, device=DEV)
                     for kind in dict.fromkeys(kinds)]
        at, outs = {}, []
        for k, kind in zip(sizes, kinds):
            buf = s["flat"][list(dict.fromkeys(kinds)).index(kind)]
            outs.append(buf[at.get(kind, 0):at.get(kind, 0) + k])
            at[kind] = at.get(kind, 0) + k
        s["outs"] = outs
    elif case["op"] in ("norm", "norm8"):
        n, dim, dt, pad = case["n"], case["dim"], TYPES[case["dtype"]], case["pad"]
        x = torch.randn((n, dim + pad), generator=g, device=DEV)
        x[:, :dim] *= _spread(g, dim)
        s["x"] = x.to(dt)[:, :dim]
        # the coarser stage's features are larger than the finer one's
        s["residual"] = (2.0 * _randn(g, (n, dim), torch.float32)).to(dt) if case["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn(dim, generator=g, device=DEV)).to(dt) if case["affine"] else None
        if case["op"] == "norm":
            s["dy"] = _randn(g, (n, dim), dt, pad)
            s["dsum"] = _randn(g, (n, dim), dt) if case["residual"] else None
    elif case["op"] == "quant":
        n, dim, dt, pad = case["n"], case["dim"], TYPES[case["dtype"]], case["pad"]
        x = torch.randn((n, dim + pad), generator=g, device=DEV) / math.sqrt(dim)
        x[:, :dim] *= _spread(g, dim)
        s["x"] = x.to(dt)[:, :dim]
    else:
        n, dim, vocab = case["n"], case["dim"], case["vocab"]
        # normalised features and a vocabulary as the label head starts with, both in 8 bits
        s["q"], s["q_scales"] = _quantize(_randn(g, (n, dim), torch.float32))
        s["w"], s["w_scales"] = _quantize(_randn(g, (vocab, dim), torch.float32) * _spread(g, dim) / math.sqrt(dim))
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """What a program keeps: outputs, workspaces, and the clipping's handle of its gradient buffers."""
    from differentiable_gaussian_splat_amd import labels as L
    from differentiable_gaussian_splat_amd import optim as O

    c = s["case"]
    empty = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=DEV)
    if c["op"] == "clip":
        s["clip"] = O.GradClip(s["grads"], s["outs"])  # a training loop's gradient buffers stay the same
        return
    n, dim, dt = c["n"], c["dim"], TYPES[c["dtype"]]
    if c["op"] == "norm":
        s["h"] = empty(n, dim, dtype=dt) if c["residual"] else None
        s["y"], s["dx"], s["rstd"] = empty(n, dim, dtype=dt), empty(n, dim, dtype=dt), empty(n, dtype=torch.float32)
        s["dweight"] = empty(dim, dtype=dt) if c["affine"] else None
        s["ws"] = empty(L.gs_rms_norm_bwd_workspace_size(n, dim, dt), dtype=torch.uint8)
    elif c["op"] == "norm8":
        s["h"] = empty(n, dim, dtype=dt) if c["residual"] else None
        s["q"], s["scales"] = L.rows_q8(n, dim, DEV)
    elif c["op"] == "quant":
        s["q"], s["scales"] = L.rows_q8(n, dim, DEV)
    else:
        s["out"] = empty(n, c["vocab"], dtype=dt)


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from differentiable_gaussian_splat_amd import labels as L

    op = s["case"]["op"]
    if op == "clip":
        return dict(norm=s["clip"](s["max_norm"]), out=s["flat"])
    if op == "norm":
        L.gs_rms_norm_fwd(s["x"], s["weight"], s["y"], s["residual"], s["h"], s["rstd"], EPS)
        h = s["x"] if s["h"] is None else s["h"]
        L.gs_rms_norm_bwd(h, s["weight"], s["rstd"], s["dy"], s["dx"], s["dweight"], s["ws"], s["dsum"])
        return dict(y=s["y"], h=s["h"], dx=s["dx"], dweight=s["dweight"])
    if op == "norm8":
        L.gs_rms_norm_q8(s["x"], s["weight"], s["q"], s["scales"], s["residual"], s["h"], EPS)
        return dict(q=s["q"], scales=s["scales"], h=s["h"])
    if op == "quant":
        L.gs_quantize_q8(s["x"], s["q"], s["scales"])
        return dict(q=s["q"], scales=s["scales"])
    L.gs_label_scores_q8(s["q"], s["q_scales"], s["w"], s["w_scales"], s["out"])
    return dict(out=s["out"])


def _quantize(v):
    """Rows v (float32) in 8 bits: values and scales."""
    n, dim = v.shape
    cols, groups = _padded(dim)
    b = torch.nn.functional.pad(v, (0, cols - dim)).reshape(n, cols // BLOCK, BLOCK)
    m, e = torch.frexp(b.abs().amax(2))  # m 2^e with m in [0.5, 1), or 0
    e = torch.where(m == 0, 0, (e - 9 + (m > MAX8 / 512).int()).clamp(min=-126))
    q = torch.ldexp(b, -e[..., None]).to(Q8).reshape(n, cols)
    e = torch.nn.functional.pad(e, (0, groups - e.shape[1]))  # 2^0 behind the blocks
    return q, torch.ldexp(torch.ones(e.shape, device=DEV), e).to(E8)


def _dequantize(q, scales):
    """The float32 values that rows in 8 bits stand for."""
    n, cols = q.shape
    return (q.float().reshape(n, cols // BLOCK, BLOCK) * scales.float()[:, :cols // BLOCK, None]).reshape(n, cols)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "clip":
        total = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
        f = (s["max_norm"] / (total + 1e-6)).clamp(max=1.0).float()
        flat = [torch.cat([(g.float() * f).to(b.dtype) for g in s["grads"] if g.dtype is b.dtype]) for b in s["flat"]]
        return dict(norm=total.float().reshape(1), out=flat)
    if c["op"] == "scores":
        return dict(out=(_dequantize(s["q"], s["q_scales"]) @ _dequantize(s["w"], s["w_scales"]).t())
                    .to(TYPES[c["dtype"]]))
    dt = TYPES[c["dtype"]]
    x = s["x"].float()
    if c["op"] == "quant":
        q, scales = _quantize(x)
        return dict(q=q, scales=scales)
    h = (x + s["residual"].float()).to(dt) if c["residual"] else None
    x = h.float() if c["residual"] else x
    w = s["weight"].float() if c["affine"] else 1.0
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    xh = x * rstd
    if c["op"] == "norm8":
        q, scales = _quantize(xh * w)
        return dict(q=q, scales=scales, h=h)
    dy = s["dy"].float()
    g = dy * w
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    dx = dx + s["dsum"].float() if c["residual"] else dx
    return dict(y=(xh * w).to(dt), h=h, dx=dx.to(dt), dweight=(dy * xh).sum(0).to(dt) if c["affine"] else None)


# ------------------------------------------------------------------ floors and exact values

def work(case):
    if case["op"] == "clip":
        sizes = _sizes(case)
        each = {"f32": [4], "bf16": [2], "both": [4, 2]}[case["dtype"]]
        return dict(bytes=sum(2 * k * each[i % len(each)] for i, k in enumerate(sizes)) + 4, flops=3 * sum(sizes))
    n, dim, size = case["n"], case["dim"], 4 if case["dtype"] == "f32" else 2
    cols, groups = _padded(dim)
    if case["op"] == "scores":
        return dict(bytes=(n + case["vocab"]) * (cols + groups) + n * case["vocab"] * size,
                    flops=2 * n * dim * case["vocab"])
    if case["op"] == "quant":
        return dict(bytes=n * dim * size + n * (cols + groups), flops=3 * n * dim)
    par, matrices = dim * size if case["affine"] else 0, 3 if case["residual"] else 1
    if case["op"] == "norm8":  # x, the residual, their sum
        return dict(bytes=matrices * n * dim * size + par + n * (cols + groups), flops=8 * n * dim)
    # x, y, dy, dx; the residual, the sum and its gradient
    return dict(bytes=(3 + (4 if case["residual"] else 1)) * n * dim * size + 2 * par, flops=18 * n * dim)


def exact(case, seed):
    """The same outputs in 64 bits from the definitions (the norm's gradient through its projection, products block by
    block); rows in 8 bits as the quotients before their rounding."""
    global own
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    d = torch.float64
    if case["op"] == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.to(d))) ** 2 for g in s["grads"]))
        f = min(1.0, s["max_norm"] / (norm + 1e-6))
        return dict(norm=torch.full((1,), norm, dtype=d, device=DEV),
                    out=[torch.cat([g for g in s["grads"] if g.dtype is b.dtype]).to(d) * f for b in s["flat"]])
    if case["op"] == "scores":
        out = torch.zeros((case["n"], case["vocab"]), dtype=d, device=DEV)
        for b in range(s["q"].shape[1] // BLOCK):
            cols = slice(b * BLOCK, (b + 1) * BLOCK)
            out.addmm_(s["q"][:, cols].to(d) * s["q_scales"][:, b:b + 1].to(d),
                       (s["w"][:, cols].to(d) * s["w_scales"][:, b:b + 1].to(d)).t())
        return dict(out=out)
    x = s["x"].to(d)
    if case["op"] == "quant":
        return _exact_rows(x)
    h = None
    if case["residual"]:
        h = x + s["residual"].to(d)
        x = h.to(TYPES[case["dtype"]]).to(d)  # the norm is of the sum that is handed on
    w = s["weight"].to(d) if case["affine"] else torch.ones(case["dim"], dtype=d, device=DEV)
    rstd = 1.0 / torch.sqrt(torch.linalg.vector_norm(x, dim=1) ** 2 / case["dim"] + EPS)
    xh = x * rstd[:, None]
    if case["op"] == "norm8":
        return dict(_exact_rows(xh * w), h=h)
    dy = s["dy"].to(d)
    # dx = rstd (I - xh xh^T / dim) (w dy)
    g = dy * w
    dx = torch.addcmul(g, xh, torch.einsum("ij,ij->i", g, xh)[:, None], value=-1.0 / case["dim"]) * rstd[:, None]
    if case["residual"]:
        dx += s["dsum"].to(d)
    return dict(y=xh * w, h=h, dx=dx, dweight=torch.einsum("ij,ij->j", dy, xh) if case["affine"] else None)


def _exact_rows(v):
    """Quotients and scales of rows v in 64 bits."""
    n, dim = v.shape
    cols, groups = _padded(dim)
    q = torch.zeros((n, cols), dtype=torch.float64, device=DEV)
    scales = torch.ones((n, groups), dtype=torch.float64, device=DEV)
    for b in range(cols // BLOCK):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        top = torch.linalg.vector_norm(part, ord=math.inf, dim=1)
        e = torch.where(top > 0, torch.ceil(torch.log2(top / MAX8)), 0.0).clamp(min=-126.0)
        # the logarithm is off by its rounding next to a power of two
        e = torch.where(top > MAX8 * torch.exp2(e), e + 1, e)
        e = torch.where((top > 0) & (e > -126) & (top <= MAX8 * torch.exp2(e - 1)), e - 1, e)
        scales[:, b] = torch.exp2(e)
        q[:, b * BLOCK:b * BLOCK + part.shape[1]] = part / torch.exp2(e)[:, None]
    return dict(q=q, scales=scales)
