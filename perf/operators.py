"""Timed cases of the label-learning operators of ``differentiable_gaussian_splat_amd.labels``.

Three operators that together learn labels of a scene's Gaussians (or of
rendered pixels): the lookup of a feature codebook by each Gaussian's code
with its gradient, layer normalisation of the features with its gradients, and
the softmax cross entropy of the normalised features against a vocabulary of
labels with its gradients.

    embed   out[i] = scale table[ids[i]], a zero row where ids[i] names no row;
            dtable[v] = scale sum_{i: ids[i] = v} dout[i]
    norm    y = (x - mean) rstd weight + bias, statistics over the columns;
            dx, dweight, dbias
    loss    loss[i] = log sum_v exp(x[i] . w[v]) - x[i] . w[labels[i]], zero where
            labels[i] names no label; mean = sum loss / max(labelled rows, 1);
            dx, dw of the mean, or of sum_i dloss[i] loss[i]

With ``own`` false, ``run`` is the plain form: elementary torch operations in
float32, rounded once at the end. With ``own`` true it makes the library's
calls.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


# ------------------------------------------------------------------ cases

def _embed(n, dim, vocab, dtype, grad, skew, missing, pad=0, wide=False):
    return dict(op="embed", n=n, dim=dim, vocab=vocab, dtype=dtype, grad=grad, skew=skew, missing=missing, pad=pad,
                wide=wide)


def _norm(n, dim, dtype, grad, affine=True, pad=0):
    return dict(op="norm", n=n, dim=dim, dtype=dtype, grad=grad, affine=affine, pad=pad)


def _loss(n, dim, vocab, dtype, grad, missing, rows=False, wide=False):
    return dict(op="loss", n=n, dim=dim, vocab=vocab, dtype=dtype, grad=grad, missing=missing, rows=rows, wide=wide)


def listed():
    return [
        # a handful of picked Gaussians: launch latency is all there is
        dict(_embed(33, 32, 500, "f32", True, 0.0, 0.0), name="embed_pick"),
        # every Gaussian of a million-Gaussian scene into a 16384-row feature codebook
        dict(_embed(1_000_000, 64, 16_384, "f32", True, 1.0, 0.02), name="embed_scene"),
        # tokens of label texts: wide rows of a large table, a few words in most of them
        dict(_embed(65_536, 512, 65_536, "bf16", True, 1.6, 0.0, wide=True), name="embed_text"),
        # an odd row length in the columns of a wider matrix, a tenth of the Gaussians without a code
        dict(_embed(200_003, 27, 4_099, "f32", True, 0.5, 0.1, pad=5), name="embed_odd"),
        # the features of a picked region, inference
        dict(_norm(64, 64, "f32", False), name="norm_pick"),
        # one feature vector per Gaussian of a million-Gaussian scene, a training step
        dict(_norm(1_000_000, 64, "f32", True), name="norm_scene"),
        # wide features of a batch of pixels, a training step
        dict(_norm(32_768, 1024, "bf16", True), name="norm_wide"),
        # odd row length in the columns of a wider matrix, a training step
        dict(_norm(7_777, 771, "bf16", True, pad=6), name="norm_odd"),
        # a few labelled Gaussians against a closed label set, a training step
        dict(_loss(48, 32, 1_000, "f32", True, 0.1, wide=True), name="loss_pick"),
        # a float32 head on partly labelled Gaussians, weighted rows, odd sizes
        dict(_loss(5_003, 129, 8_191, "f32", True, 0.3, rows=True), name="loss_partial"),
        # scoring a batch of pixels against an open vocabulary, no gradient
        dict(_loss(8_192, 256, 50_021, "bf16", False, 0.05), name="loss_score"),
        # training an open-vocabulary head on wide features: the largest product
        dict(_loss(8_192, 1024, 65_536, "bf16", True, 0.0), name="loss_vocab"),
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
    op = rng.choice(["embed", "norm", "loss"])
    dtype = rng.choice(["f32", "bf16"])
    grad = rng.random() < 0.75
    if op == "embed":
        n, dim = _size(rng, 1, 1_000_000), _size(rng, 1, 1024)
        n = max(1, min(n, 64_000_000 // dim))
        vocab = max(1, min(_size(rng, 2, 131_072), 64_000_000 // dim))
        return _embed(n, dim, vocab, dtype, grad, rng.choice([0.0, 0.5, 1.0, 1.6]), rng.choice([0.0, 0.02, 0.3]),
                      pad=rng.choice([0, 0, 3, 8]), wide=rng.random() < 0.5)
    if op == "norm":
        n, dim = _size(rng, 1, 1_000_000), _size(rng, 1, 8192)
        n = max(1, min(n, 64_000_000 // dim))
        return _norm(n, dim, dtype, grad, affine=rng.random() < 0.8, pad=rng.choice([0, 0, 3, 8]))
    n, dim, vocab = _size(rng, 1, 65_536), _size(rng, 8, 1024), _size(rng, 2, 131_072)
    # products of at most a quarter of the largest listed case in float32, all of it in bfloat16
    most = 8_192 * 1024 * 65_536 // (4 if dtype == "f32" else 1)
    vocab = max(2, min(vocab, most // (n * dim), (1 << 30) // n))
    return _loss(n, dim, vocab, dtype, grad, rng.choice([0.0, 0.1, 0.6, 1.0 if n < 100 else 0.9]),
                 rows=rng.random() < 0.4, wide=rng.random() < 0.5)


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


def _codes(g, n, vocab, skew, missing, wide):
    """Row numbers below vocab: rank r drawn with weight near r^-skew, ranks
    scattered over the rows; a share of them -1."""
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    if skew == 0.0:
        r = u * vocab
    elif skew == 1.0:
        r = torch.exp(u * math.log(vocab + 1.0)) - 1.0
    else:
        a = 1.0 - skew
        r = (1.0 + u * ((vocab + 1.0) ** a - 1.0)) ** (1.0 / a) - 1.0
    r = r.to(torch.int64).clamp_(0, vocab - 1)
    rows = torch.randperm(vocab, generator=g, device=DEV)
    ids = rows[r]
    if missing:
        ids = torch.where(torch.rand(n, generator=g, device=DEV) < missing, -1, ids)
    return ids if wide else ids.to(torch.int32)


def prepare(case, seed):
    n, dim, dt = case["n"], case["dim"], TYPES[case["dtype"]]
    g = _gen(seed, 17)
    s = dict(case=case)
    if case["op"] == "embed":
        s["table"] = _randn(g, (case["vocab"], dim), dt, case["pad"])
        s["ids"] = _codes(g, n, case["vocab"], case["skew"], case["missing"], case["wide"])
        s["scale"] = math.sqrt(dim)
        if case["grad"]:
            s["dout"] = (_randn(g, (n, dim), torch.float32, case["pad"]) / 64).to(dt)
    elif case["op"] == "norm":
        # features with a column-dependent offset and spread, as learned ones have
        spread = torch.exp(0.5 * torch.randn(dim, generator=g, device=DEV))
        offset = 0.5 * torch.randn(dim, generator=g, device=DEV)
        wide = torch.randn((n, dim + case["pad"]), generator=g, device=DEV)
        wide[:, :dim] = wide[:, :dim] * spread + offset
        s["x"] = wide.to(dt)[:, :dim]
        s["weight"] = s["bias"] = None
        if case["affine"]:
            s["weight"] = (1 + 0.2 * torch.randn(dim, generator=g, device=DEV)).to(dt)
            s["bias"] = (0.2 * torch.randn(dim, generator=g, device=DEV)).to(dt)
        if case["grad"]:
            s["dy"] = _randn(g, (n, dim), dt, case["pad"])
    else:
        vocab = case["vocab"]
        s["labels"] = _codes(g, n, vocab, 1.0, case["missing"], case["wide"])
        s["w"] = (_randn(g, (vocab, dim), torch.float32) / math.sqrt(dim)).to(dt)
        # normalised features leaning towards their label, as in a head half way through its training
        x = _randn(g, (n, dim), torch.float32)
        x = x + 2.0 * s["w"][s["labels"].clamp(min=0).long()].float()
        s["x"] = x.to(dt)
        if case["grad"]:
            if case["rows"]:
                s["dloss"] = torch.rand(n, generator=g, device=DEV) / n
            else:
                s["dmean"] = torch.ones(1, device=DEV)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The buffers that a program keeps: outputs and workspaces."""
    from differentiable_gaussian_splat_amd import labels as L

    c = s["case"]
    n, dim, dt = c["n"], c["dim"], TYPES[c["dtype"]]
    empty = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device=DEV)
    if c["op"] == "embed":
        s["out"] = empty(n, dim)
        if c["grad"]:
            s["dtable"] = empty(c["vocab"], dim)
            s["ws"] = empty(L.gs_embed_bwd_workspace_size(n, dim, c["vocab"], dt), dtype=torch.uint8)
    elif c["op"] == "norm":
        s["y"] = empty(n, dim)
        s["mean"], s["rstd"] = empty(n, dtype=torch.float32), empty(n, dtype=torch.float32)
        if c["grad"]:
            s["dx"] = empty(n, dim)
            s["dweight"] = empty(dim) if c["affine"] else None
            s["dbias"] = empty(dim) if c["affine"] else None
            s["ws"] = empty(L.gs_layer_norm_bwd_workspace_size(n, dim, dt), dtype=torch.uint8)
    else:
        s["loss"], s["lse"] = empty(n, dtype=torch.float32), empty(n, dtype=torch.float32)
        s["mean"], s["count"] = empty(1, dtype=torch.float32), empty(1, dtype=torch.int32)
        s["ws"] = empty(L.gs_label_loss_workspace_size(n, dim, c["vocab"], dt, c["grad"]), dtype=torch.uint8)
        if c["grad"]:
            s["dx"], s["dw"] = empty(n, dim), empty(c["vocab"], dim)


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from differentiable_gaussian_splat_amd import labels as L

    c = s["case"]
    if c["op"] == "embed":
        L.gs_embed_fwd(s["table"], s["ids"], s["out"], s["scale"])
        if not c["grad"]:
            return dict(out=s["out"])
        L.gs_embed_bwd(s["ids"], s["dout"], s["dtable"], s["ws"], s["scale"])
        return dict(out=s["out"], dtable=s["dtable"])
    if c["op"] == "norm":
        L.gs_layer_norm_fwd(s["x"], s["weight"], s["bias"], s["y"], s["mean"], s["rstd"], EPS)
        if not c["grad"]:
            return dict(y=s["y"], mean=s["mean"], rstd=s["rstd"])
        L.gs_layer_norm_bwd(s["x"], s["weight"], s["mean"], s["rstd"], s["dy"], s["dx"], s["dweight"], s["dbias"],
                            s["ws"])
        out = dict(y=s["y"], dx=s["dx"])
        if c["affine"]:
            out.update(dweight=s["dweight"], dbias=s["dbias"])
        return out
    L.gs_label_loss_fwd(s["x"], s["w"], s["labels"], s["loss"], s["lse"], s["mean"], s["count"], s["ws"])
    out = dict(loss=s["loss"], mean=s["mean"], count=s["count"])
    if not c["grad"]:
        return dict(out, lse=s["lse"])
    L.gs_label_loss_bwd(s["x"], s["w"], s["labels"], s["lse"], s["dx"], s["dw"], s["ws"], dmean=s.get("dmean"),
                        dloss=s.get("dloss"))
    return dict(out, dx=s["dx"], dw=s["dw"])


def _run_plain(s):
    c = s["case"]
    dt = TYPES[c["dtype"]]
    if c["op"] == "embed":
        ids = s["ids"].long()
        have = ids >= 0
        out = s["table"].float()[ids.clamp(min=0)] * s["scale"]
        out = torch.where(have[:, None], out, 0.0).to(dt)
        if not c["grad"]:
            return dict(out=out)
        # one row more for the rows without a code; they are sorted so that equal rows add up in order
        order = torch.argsort(torch.where(have, ids, c["vocab"]), stable=True)
        rows = torch.where(have, ids, c["vocab"])[order]
        dtable = torch.zeros((c["vocab"] + 1, c["dim"]), dtype=torch.float32, device=DEV)
        dtable.index_add_(0, rows, s["dout"].float()[order] * s["scale"])
        return dict(out=out, dtable=dtable[:-1].to(dt))
    if c["op"] == "norm":
        x = s["x"].float()
        w = s["weight"].float() if c["affine"] else 1.0
        b = s["bias"].float() if c["affine"] else 0.0
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = torch.rsqrt((xc * xc).mean(1, keepdim=True) + EPS)
        xh = xc * rstd
        y = (xh * w + b).to(dt)
        if not c["grad"]:
            return dict(y=y, mean=mean[:, 0], rstd=rstd[:, 0])
        dy = s["dy"].float()
        g = dy * w
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        out = dict(y=y, dx=dx.to(dt))
        if c["affine"]:
            out.update(dweight=(dy * xh).sum(0).to(dt), dbias=dy.sum(0).to(dt))
        return out
    x, w, lab = s["x"].float(), s["w"].float(), s["labels"].long()
    have = lab >= 0
    count = have.sum()
    logits = x @ w.t()
    top = logits.max(1, keepdim=True).values
    e = torch.exp(logits - top)
    z = e.sum(1, keepdim=True)
    lse = (top + torch.log(z))[:, 0]
    hit = lab.clamp(min=0)[:, None]
    loss = torch.where(have, lse - logits.gather(1, hit)[:, 0], 0.0)
    lse = torch.where(have, lse, 0.0)
    mean = loss.sum(dtype=torch.float64) / count.clamp(min=1)
    out = dict(loss=loss, mean=mean.float().reshape(1), count=count.to(torch.int32).reshape(1))
    if not c["grad"]:
        return dict(out, lse=lse)
    del logits
    up = s["dloss"] if c["rows"] else (s["dmean"] / count.clamp(min=1)).expand(c["n"])
    up = torch.where(have, up, 0.0)[:, None]
    e.div_(z)
    e.scatter_add_(1, hit, torch.full_like(z, -1.0))
    e.mul_(up)
    return dict(out, dx=(e @ w).to(dt), dw=(e.t() @ x).to(dt))


# ------------------------------------------------------------------ floors and exact values

def work(case):
    n, dim, size = case["n"], case["dim"], 4 if case["dtype"] == "f32" else 2
    if case["op"] == "embed":
        idx = n * (8 if case["wide"] else 4)
        table = min(case["vocab"], n) * dim * size  # rows that can be read
        b = idx + table + n * dim * size
        f = n * dim
        if case["grad"]:
            b += n * dim * size + case["vocab"] * dim * size
            f += 2 * n * dim
        return dict(bytes=b, flops=f)
    if case["op"] == "norm":
        par = 2 * dim * size if case["affine"] else 0
        b, f = 2 * n * dim * size + par, 8 * n * dim
        if case["grad"]:
            b += 2 * n * dim * size + par
            f += 14 * n * dim
        else:
            b += 8 * n
        return dict(bytes=b, flops=f)
    vocab = case["vocab"]
    b = (n * dim + vocab * dim) * size + n * (8 if case["wide"] else 4) + 4 * n
    f = 2 * n * dim * vocab
    if case["grad"]:
        b += (n * dim + vocab * dim) * size
        f *= 3
    return dict(bytes=b, flops=f)


def exact(case, seed):
    """The same outputs in 64 bits from the definitions (the loss by rows of the
    vocabulary's products, the normalisation's gradient through its projection,
    the table's gradient by running sums over the sorted codes)."""
    if case["op"] == "loss" and (6 if case["grad"] else 2) * case["n"] * case["dim"] * case["vocab"] > 3e14:
        return None  # beyond about 20 seconds of 64-bit products
    global own
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    d = torch.float64
    if case["op"] == "embed":
        ids = s["ids"].long()
        table = torch.cat([s["table"].to(d), torch.zeros((1, case["dim"]), dtype=d, device=DEV)])
        slot = torch.where(ids < 0, case["vocab"], ids)
        res = dict(out=table.index_select(0, slot) * s["scale"])
        if case["grad"]:
            order = torch.argsort(slot)
            counts = torch.bincount(slot, minlength=case["vocab"] + 1)
            dtable = torch.zeros((case["vocab"], case["dim"]), dtype=d, device=DEV)
            ends = torch.cumsum(counts, 0)
            for c0 in range(0, case["dim"], 16):  # columns at a time: the sums need a row per token
                cols = s["dout"][:, c0:c0 + 16].to(d)[order]
                run_ = torch.cat([torch.zeros((1, cols.shape[1]), dtype=d, device=DEV), torch.cumsum(cols, 0)])
                dtable[:, c0:c0 + 16] = (run_[ends] - run_[ends - counts])[:-1]
            res["dtable"] = dtable * s["scale"]
        return res
    if case["op"] == "norm":
        x = s["x"].to(d)
        w = s["weight"].to(d) if case["affine"] else torch.ones(case["dim"], dtype=d, device=DEV)
        b = s["bias"].to(d) if case["affine"] else torch.zeros(case["dim"], dtype=d, device=DEV)
        mean = x.sum(1) / case["dim"]
        xh = x - mean[:, None]
        rstd = 1.0 / torch.sqrt(torch.linalg.vector_norm(xh, dim=1) ** 2 / case["dim"] + EPS)
        xh *= rstd[:, None]
        res = dict(y=torch.addcmul(b, xh, w))
        if not case["grad"]:
            return dict(res, mean=mean, rstd=rstd)
        dy = s["dy"].to(d)
        # dx = rstd (I - (1 1^T + xh xh^T) / dim) (w dy)
        g = dy * w
        res["dx"] = (g - (torch.einsum("ij->i", g)[:, None] + xh * torch.einsum("ij,ij->i", g, xh)[:, None])
                     / case["dim"]) * rstd[:, None]
        if case["affine"]:
            res.update(dweight=torch.einsum("ij,ij->j", dy, xh), dbias=torch.einsum("ij->j", dy))
        return res
    x, w, lab = s["x"].to(d), s["w"].to(d), s["labels"].long()
    kept = torch.nonzero(lab >= 0)[:, 0]
    count = kept.numel()
    loss = torch.zeros(case["n"], dtype=d, device=DEV)
    lse = torch.zeros(case["n"], dtype=d, device=DEV)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    if case["grad"]:
        up = s["dloss"].to(d) if case["rows"] else torch.full((case["n"],), float(s["dmean"]) / max(count, 1), dtype=d,
                                                              device=DEV)
    step = max(1, (1 << 28) // case["vocab"])
    for k0 in range(0, count, step):
        r = kept[k0:k0 + step]
        z = torch.mm(x[r], w.t())
        l = torch.logsumexp(z, 1)
        lse[r] = l
        loss[r] = l - z[torch.arange(r.numel(), device=DEV), lab[r]]
        if case["grad"]:
            p = torch.softmax(z, 1)
            p[torch.arange(r.numel(), device=DEV), lab[r]] -= 1.0
            p *= up[r][:, None]
            dx[r] = torch.mm(p, w)
            dw += torch.mm(p.t(), x[r])
    res = dict(loss=loss, mean=loss.sum().reshape(1) / max(count, 1),
               count=torch.full((1,), count, dtype=torch.int32, device=DEV))
    if case["grad"]:
        return dict(res, dx=dx, dw=dw)
    return dict(res, lse=lse)
