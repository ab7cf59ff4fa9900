"""Measured cases of a block over the rows of segments: seg_layer_norm (rows
normalised, scaled and shifted by their segment's own weight and bias, or by
shared ones) and seg_gated (the gated feed-forward block: both projections of a
segment's rows, the activation of the first and the product), each forward
alone, as it is served, and forward and backward, as it is trained.

Segments are offset-delimited: rows [offsets[s], offsets[s+1]) of x belong to
segment s.  A row in no segment gives 0 and has the gradient 0.  The plain
products work on chunks: every segment's rows are cut into chunks of C rows
(the last one padded), each chunk is one batch entry of a batched product with
its segment's matrix.  Nothing is read back to the host.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
# (not relu, whose derivative jumps: a product next to 0 would decide what a gradient is)
ACTIVATIONS = ("silu", "gelu", "gelu_tanh", "sigmoid")
EPS = 1e-5
MAX_FLOPS = 1.65e12     # of a drawn gated case: the largest listed one's
MAX_VALUES = 7.0e7      # rows x columns of a drawn norm: the largest listed one's
MAX_PLAIN = 3.0e9       # values that the plain form's gathered matrices may hold


def _gated(name, dtype, rows, segments, k, n, step=False, act="silu", trans=False, spread=0.4, pad=0):
    """n columns of each projection; step: forward and backward."""
    return {"name": name, "op": "gated", "dtype": dtype, "rows": rows, "segments": segments, "k": k, "n": n, "step": step,
            "act": act, "trans": trans, "spread": spread, "pad": pad}


def _norm(name, dtype, rows, segments, k, step=False, wt="same", bias=True, spread=0.4, pad=0):
    """k columns; segments 0: one weight and bias for all rows; wt: the weights' type, x's or f32."""
    return {"name": name, "op": "norm", "dtype": dtype, "rows": rows, "segments": segments, "k": k, "step": step, "wt": wt,
            "bias": bias, "spread": spread, "pad": pad}


def listed():
    return [
        # one token sent to 2 of 8 experts: latency, and reading two experts' matrices
        _gated("gated one token", "bf16", 2, 8, 2048, 1024),
        # a decode step of 64 tokens, 2 of 64 experts each, matrices stored [2 N, K]: bound by the matrices
        _gated("gated decode", "bf16", 128, 64, 2048, 1024, trans=True, spread=0.8),
        # a short prompt over few, unevenly loaded experts, with unused rows at the end
        _gated("gated prompt", "f16", 4100, 16, 1024, 2048, act="gelu", trans=True, spread=1.0, pad=61),
        # a training step over evenly loaded experts
        _gated("gated train", "bf16", 32768, 32, 2048, 2048, step=True, spread=0.3),
        # a small, uneven training step of odd sizes
        _gated("gated train uneven", "f16", 5003, 64, 520, 333, step=True, act="gelu_tanh", spread=1.0, pad=5),
        # message passing (the benchmark's 1,000,000 x 64) gated by relation type, trained
        _gated("gated relations", "f32", 1000000, 50, 64, 64, step=True, act="sigmoid", spread=1.2),
        # one token: latency
        _norm("norm one token", "bf16", 1, 0, 2048),
        # a prompt, the weights kept in 32 bits
        _norm("norm prompt", "bf16", 4100, 0, 4096, wt="f32"),
        # a training step
        _norm("norm train", "bf16", 32768, 0, 2048, step=True, wt="f32", spread=0.3),
        # a training step with a norm for every expert, uneven loads
        _norm("norm experts", "f16", 20011, 64, 1000, step=True, spread=1.0, pad=61),
        # message passing, a norm for every relation type, trained
        _norm("norm relations", "f32", 1000000, 50, 64, step=True, spread=1.2),
        # few wide rows, no bias, trained
        _norm("norm wide", "bf16", 513, 0, 12288, step=True, wt="f32", bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A number of columns: mostly a multiple of 8, sometimes any."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.15 else max(8, v // 8 * 8)


def draw(rng):
    while True:
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        pad = rng.choice((0, 0, rng.randint(1, 60)))
        spread = round(rng.uniform(0.1, 1.3), 2)
        step = rng.random() < 0.5
        if rng.random() < 0.5:
            k = _width(rng, 16, 16384)
            segments = 0 if rng.random() < 0.5 else _log(rng, 1, 200)
            c = _norm("", dtype, _log(rng, 1, 1000000), segments, k, step, rng.choice(("same", "f32")), rng.random() < 0.75, spread,
                      pad if segments else 0)
            del c["name"]
            if (c["rows"] + c["pad"]) * k <= MAX_VALUES:
                return c
            continue
        narrow = dtype == "f32" and rng.random() < 0.6
        top = 160 if narrow else 2048
        rows = _log(rng, 1, 1000000 if narrow else 32768)
        c = _gated("", dtype, rows, _log(rng, 1, 128), _width(rng, 32, top), _width(rng, 32, top), step, rng.choice(ACTIVATIONS),
                   rng.random() < 0.5, spread, pad)
        del c["name"]
        chunks, size = _chunks(c)
        flops = work(c)["flops"]
        if flops <= MAX_FLOPS and flops * max(rows, chunks * size) / rows <= 2 * MAX_FLOPS and chunks * 2 * c["k"] * c["n"] <= MAX_PLAIN:
            return c


def _chunks(case):
    """(number of chunks that always suffices, rows of a chunk) of the plain products."""
    rows, segments = case["rows"], case["segments"]
    if rows <= segments:
        return rows, 1
    size = 1
    while size < 256 and size * segments < 2 * rows:
        size *= 2
    return rows // size + segments, size


def _lengths(case, rng):
    """Rows of each segment: multinomial over log-normal shares; with 8 segments or more about one in ten has none."""
    rows, segments = case["rows"], case["segments"]
    share = np.exp(rng.standard_normal(segments) * case["spread"])
    if segments >= 8:
        share[rng.random(segments) < 0.1] = 0.0
        share[int(rng.integers(segments))] += 0.5
    return rng.multinomial(rows, share / share.sum())


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, mean=0.0, dtype=dtype):
        t = torch.empty(shape, dtype=dtype, device="cuda")
        return t.normal_(mean, scale, generator=g)

    k, segments, rows = case["k"], case["segments"], case["rows"] + case["pad"]
    state = {"case": case, "offsets": None}
    if segments > 0:
        lengths = _lengths(case, rng)
        state["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)).cuda()
    if case["op"] == "gated":
        n = case["n"]
        state["x"] = normal(rows, k)
        state["w"] = normal(*((segments, 2 * n, k) if case["trans"] else (segments, k, 2 * n)), scale=k ** -0.5)
        if case["step"]:
            state["dy"] = normal(rows, n, scale=0.1)
        return state
    # activations have a mean of their own
    state["x"] = normal(rows, k, scale=1.5, mean=float(rng.uniform(-0.5, 0.5)))
    shape = (segments, k) if segments > 0 else (k,)
    wt = torch.float32 if case["wt"] == "f32" else dtype
    state["weight"] = normal(*shape, scale=0.1, mean=1.0, dtype=wt)
    state["bias"] = normal(*shape, scale=0.1, dtype=wt) if case["bias"] else None
    if case["step"]:
        state["dy"] = normal(rows, k, scale=0.1)
    return state


def _cut(case, offsets, rows):
    """The chunks of the plain products: (segment of each chunk, rows of each chunk [chunks, C], which of them are real)."""
    count, size = _chunks(case)
    each = (offsets[1:] - offsets[:-1] + size - 1) // size          # chunks of each segment
    ends = torch.cumsum(each, 0)
    i = torch.arange(count, device=offsets.device)
    seg = torch.searchsorted(ends, i, right=True)
    real = seg < offsets.numel() - 1
    seg = seg.clamp(max=offsets.numel() - 2)
    first = offsets[seg] + (i - (ends - each)[seg]) * size
    row = first[:, None] + torch.arange(size, device=offsets.device)
    real = real[:, None] & (row < offsets[seg + 1][:, None])
    return seg, row.clamp(0, rows - 1), real


def _activation(act, g):
    """The activation and its derivative."""
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(g * 0.5 ** 0.5))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    s = 1 / (1 + torch.exp(-g))
    return (s, s * (1 - s)) if act == "sigmoid" else (g * s, s * (1 + g * (1 - s)))


def _gated_plain(state):
    case, offsets, x = state["case"], state["offsets"], state["x"]
    n, size = case["n"], x.shape[0]
    seg, row, real = _cut(case, offsets, size)
    at, mask = row.reshape(-1), real[..., None]
    xc = x[row].float() * mask
    wc = state["w"][seg].float()
    if case["trans"]:
        wc = wc.transpose(1, 2)                                      # [chunks, K, 2 N]
    pre = torch.bmm(xc, wc)
    a, da = _activation(case["act"], pre[..., :n])
    out = torch.zeros(size, n, device=x.device)
    # rows that pad a chunk add nothing to the row they were clamped to
    h = out.index_add_(0, at, (a * pre[..., n:] * mask).flatten(0, 1)).to(x.dtype)
    if not case["step"]:
        return h
    dy = state["dy"][row].float() * mask
    dpre = torch.cat([dy * pre[..., n:] * da, dy * a], dim=-1)
    dx = torch.zeros(size, case["k"], device=x.device)
    dx.index_add_(0, at, torch.bmm(dpre, wc.transpose(1, 2)).flatten(0, 1))
    parts = torch.bmm(dpre.transpose(1, 2), xc) if case["trans"] else torch.bmm(xc.transpose(1, 2), dpre)
    dw = torch.zeros(state["w"].shape, device=x.device).index_add_(0, seg, parts)
    return h, dx.to(x.dtype), dw.to(x.dtype)


def _norm_plain(state):
    case, offsets, bias = state["case"], state["offsets"], state["bias"]
    x, weight = state["x"].float(), state["weight"].float()
    dtype, wt, segments = state["x"].dtype, state["weight"].dtype, case["segments"]
    shift = 0.0 if bias is None else bias.float()
    real = seg = None
    if segments > 0:
        row = torch.arange(x.shape[0], device=x.device)
        seg = torch.searchsorted(offsets, row, right=True) - 1
        real = ((seg >= 0) & (seg < segments))[:, None]
        seg = seg.clamp(0, segments - 1)
        weight, shift = weight[seg], 0.0 if bias is None else shift[seg]
    c = x - x.mean(-1, keepdim=True)
    rstd = (c.square().mean(-1, keepdim=True) + EPS).rsqrt()
    xhat = c * rstd
    y = xhat * weight + shift
    if real is not None:
        y = torch.where(real, y, torch.zeros_like(y))
    if not case["step"]:
        return y.to(dtype)
    dy = state["dy"].float()
    if real is not None:
        dy = dy * real
    g = dy * weight
    dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    # sums over up to a million rows

    def columns(t):
        if segments == 0:
            return t.sum(0, dtype=torch.float64).to(wt)
        return torch.zeros(segments, t.shape[1], dtype=torch.float64, device=t.device).index_add_(0, seg, t.double()).to(wt)
    out = [y.to(dtype), dx.to(dtype), columns(dy * xhat)]
    return out if bias is None else out + [columns(dy)]


def run(state):
    case, offsets = state["case"], state["offsets"]
    if not own:
        return _gated_plain(state) if case["op"] == "gated" else _norm_plain(state)
    import segmented_reduction_csr_gb300 as sr
    x = state["x"]
    if case["op"] == "gated":
        w, act, trans = state["w"], case["act"], case["trans"]
        if not case["step"]:
            return sr.seg_gated(x, w, offsets, act, transpose_w=trans)
        h, pre = sr.seg_gated(x, w, offsets, act, transpose_w=trans, with_pre=True)
        dx, dw = sr.seg_gated_grad(x, w, pre, state["dy"], offsets, act, transpose_w=trans)
        return h, dx, dw
    if not case["step"]:
        return sr.seg_layer_norm(x, state["weight"], state["bias"], offsets, eps=EPS)
    y, mean, rstd = sr.seg_layer_norm(x, state["weight"], state["bias"], offsets, eps=EPS, with_stats=True)
    dx, dweight, dbias = sr.seg_layer_norm_grad(x, state["dy"], mean, rstd, state["weight"], offsets, with_bias=case["bias"])
    return [y, dx, dweight] + ([dbias] if case["bias"] else [])


def work(case):
    rows, k, size = case["rows"], case["k"], SIZE[case["dtype"]]
    total, step = rows + case["pad"], case["step"]
    offsets = 8 * (case["segments"] + 1) if case["segments"] else 0
    if case["op"] == "gated":
        # at most `rows` matrices are needed; each gradient is written for every segment and row
        n = case["n"]
        b = size * (rows * k + min(rows, case["segments"]) * 2 * k * n + total * n) + offsets
        if step:
            b += size * (rows * n + total * k + case["segments"] * 2 * k * n)
        return {"bytes": b, "flops": (3 if step else 1) * 4.0 * rows * k * n}
    wsize = 4 if case["wt"] == "f32" else size
    weights = (2 if case["bias"] else 1) * max(1, min(case["segments"], rows)) * k * wsize
    b = size * (rows + total) * k + weights + offsets
    if step:
        b += size * (rows + total) * k + weights
    return {"bytes": b, "flops": (22.0 if step else 8.0) * rows * k}


def exact(case, seed):
    state = prepare(case, seed)
    x = state["x"].double()
    rows = x.shape[0]
    if case["segments"] > 0:
        off = state["offsets"].tolist()
        pairs = [(s, slice(off[s], off[s + 1])) for s in range(case["segments"]) if off[s + 1] > off[s]]
    else:
        pairs = [(0, slice(0, rows))]
    if case["op"] == "gated":
        n, act = case["n"], case["act"]
        h = x.new_zeros(rows, n)
        dx, dw = torch.zeros_like(x), x.new_zeros(state["w"].shape)
        for s, at in pairs:
            w = state["w"][s].double()
            w = w if case["trans"] else w.t()                        # [2 N, K]
            gate, up = x[at] @ w[:n].t(), x[at] @ w[n:].t()
            if act == "silu":
                p = torch.special.expit(gate)
                f, d = gate * p, p + gate * p * (1 - p)
            elif act == "sigmoid":
                f = torch.special.expit(gate)
                d = f * (1 - f)
            elif act == "gelu":
                p = torch.special.ndtr(gate)
                f, d = gate * p, p + gate * torch.exp(-gate.square() / 2) / math.sqrt(2 * math.pi)
            else:
                inner = math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3)
                p = torch.special.expit(2 * inner)                   # (1 + tanh(inner)) / 2
                f, d = gate * p, p + gate * 2 * p * (1 - p) * math.sqrt(2 / math.pi) * (1 + 0.134145 * gate.square())
            h[at] = f * up
            if case["step"]:
                dy = state["dy"][at].double()
                dgate, dup = dy * up * d, dy * f
                dx[at] = dgate @ w[:n] + dup @ w[n:]
                part = torch.cat([dgate.t() @ x[at], dup.t() @ x[at]])
                dw[s] = part if case["trans"] else part.t()
        return (h, dx, dw) if case["step"] else h
    weight, bias = state["weight"].double(), state["bias"]
    weight = weight.reshape(-1, case["k"])
    bias = torch.zeros_like(weight) if bias is None else bias.double().reshape(-1, case["k"])
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    dweight, dbias = torch.zeros_like(weight), torch.zeros_like(weight)
    for s, at in pairs:
        xs = x[at]
        var, mean = torch.var_mean(xs, dim=1, correction=0, keepdim=True)
        sd = torch.sqrt(var + EPS)
        z = (xs - mean) / sd
        y[at] = z * weight[s] + bias[s]
        if case["step"]:
            dy = state["dy"][at].double()
            dweight[s], dbias[s] = (dy * z).sum(0), dy.sum(0)
            dz = dy * weight[s]
            dx[at] = (dz - dz.mean(1, keepdim=True) - z * (dz * z).mean(1, keepdim=True)) / sd
    if not case["step"]:
        return y
    shape = state["weight"].shape
    out = [y, dx, dweight.reshape(shape)]
    return out + [dbias.reshape(shape)] if case["bias"] else out
