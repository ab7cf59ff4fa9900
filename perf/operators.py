"""Measured cases of the segment products: seg_matmul (rows of segment s times
the segment's own matrix), seg_matmul_grad_w (its weight gradient) and
seg_lora (a shared projection with low-rank adapters of many requests).

Segments are offset-delimited: rows [offsets[s], offsets[s+1]) of x belong to
segment s.  A row in no segment gives 0 (seg_lora: the shared product alone).
The plain forms below work on chunks: every segment's rows are cut into
chunks of C rows (the last one padded), each chunk is one batch entry of a
batched product with its segment's matrix.  Nothing is read back to the host.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
MAX_FLOPS = 5.5e11      # of a drawn case: the largest listed one's
MAX_PLAIN = 3.0e9       # values that the plain form's gathered matrices may hold


def _mm(name, dtype, rows, segments, k, n, trans=False, spread=0.4, pad=0):
    return {"name": name, "op": "mm", "dtype": dtype, "rows": rows, "segments": segments, "k": k, "n": n,
            "trans": trans, "spread": spread, "pad": pad}


def _gw(name, dtype, rows, segments, k, n, out="same", spread=0.4, pad=0):
    return {"name": name, "op": "gw", "dtype": dtype, "rows": rows, "segments": segments, "k": k, "n": n,
            "out": out, "spread": spread, "pad": pad}


def _lora(name, dtype, rows, segments, k, n, rank, adapters, spread=0.8, pad=0):
    return {"name": name, "op": "lora", "dtype": dtype, "rows": rows, "segments": segments, "k": k, "n": n,
            "rank": rank, "adapters": adapters, "spread": spread, "pad": pad}


def listed():
    return [
        # one token sent to 2 of 8 experts: latency, and reading two matrices
        _mm("mm one token", "bf16", 2, 8, 2048, 2048),
        # a decode step of 64 tokens, 2 of 64 experts each: a few rows per expert, bound by the matrices
        _mm("mm decode", "bf16", 128, 64, 2048, 1024, spread=0.8),
        # a short prompt over few, unevenly loaded experts, with unused rows at the end
        _mm("mm prompt", "f16", 4100, 16, 1024, 4096, spread=1.0, pad=61),
        # a training batch over evenly loaded experts
        _mm("mm train", "bf16", 32768, 32, 2048, 4096, spread=0.3),
        # its input gradient, with smaller matrices and uneven loads
        _mm("mm input gradient", "bf16", 20011, 64, 4096, 1024, trans=True, spread=1.0),
        # message passing: 64 features (the benchmark's shape) times a matrix per relation type
        _mm("mm relations", "f32", 1000000, 50, 64, 64, spread=1.2),
        # the weight gradient of the training batch
        _gw("gw train", "bf16", 32768, 32, 2048, 4096, spread=0.3),
        # a small batch over many experts, some without rows; 300 columns; gradients kept in 32 bits
        _gw("gw small", "f16", 700, 64, 512, 300, out="f32", spread=1.0),
        # the weight gradient of the relation types' matrices
        _gw("gw relations", "f32", 1000000, 50, 64, 64, spread=1.2),
        # one token of one request
        _lora("lora one token", "bf16", 1, 1, 2048, 2048, 16, 8),
        # a decode step of 96 requests with 64 adapters
        _lora("lora decode", "bf16", 96, 96, 4096, 4096, 16, 64),
        # prompts of 24 requests of uneven lengths
        _lora("lora prompts", "bf16", 8193, 24, 4096, 4096, 32, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A number of columns: mostly a multiple of 8, sometimes any."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.15 else max(8, v // 8 * 8)


def draw(rng):
    while True:
        op = rng.choice(("mm", "mm", "gw", "lora"))
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        pad = rng.choice((0, 0, rng.randint(1, 40)))
        spread = round(rng.uniform(0.1, 1.5), 2)
        if op == "lora":
            rows = _log(rng, 1, 12000)
            segments = rows if rng.random() < 0.4 and rows <= 512 else min(rows, _log(rng, 1, 128))
            c = _lora("", dtype, rows, segments, _width(rng, 256, 6000), _width(rng, 256, 6000),
                      rng.choice((4, 8, 8, 12, 16, 16, 32, 64)), _log(rng, 1, 64), spread, pad)
        else:
            narrow = dtype == "f32" and rng.random() < 0.6
            top = 160 if narrow else 4096
            rows = _log(rng, 1, 1000000 if narrow else 32768)
            segments, k, n = _log(rng, 1, 128), _width(rng, 32, top), _width(rng, 32, top)
            if op == "mm":
                c = _mm("", dtype, rows, segments, k, n, rng.random() < 0.5, spread, pad)
            else:
                c = _gw("", dtype, rows, segments, k, n, rng.choice(("same", "f32")), spread, pad)
        del c["name"]
        chunks, size = _chunks(c)
        values = chunks * c["k"] * c["n"] if op != "lora" else chunks * c["rank"] * (c["k"] + c["n"])
        flops = 2.0 * max(c["rows"], chunks * size if op != "lora" else 0) * c["k"] * c["n"]
        if flops <= MAX_FLOPS * 2 and work(c)["flops"] <= MAX_FLOPS and values <= MAX_PLAIN:
            return c


def _chunks(case):
    """(number of chunks that always suffices, rows of a chunk) of the plain form."""
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
    if case["op"] == "lora" and rows == segments:
        return np.ones(segments, dtype=np.int64)       # a decode step: one row each
    share = np.exp(rng.standard_normal(segments) * case["spread"])
    if case["op"] == "lora":
        return 1 + rng.multinomial(rows - segments, share / share.sum())
    if segments >= 8:
        share[rng.random(segments) < 0.1] = 0.0
        share[int(rng.integers(segments))] += 0.5
    return rng.multinomial(rows, share / share.sum())


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        t = torch.empty(shape, dtype=dtype, device="cuda")
        return t.normal_(0.0, scale, generator=g)

    k, n, segments = case["k"], case["n"], case["segments"]
    rows = case["rows"] + case["pad"]
    lengths = _lengths(case, rng)
    offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)).cuda()
    state = {"case": case, "offsets": offsets, "x": normal(rows, k)}
    if case["op"] == "mm":
        shape = (segments, n, k) if case["trans"] else (segments, k, n)
        state["w"] = normal(*shape, scale=k ** -0.5)
    elif case["op"] == "gw":
        state["dy"] = normal(rows, n, scale=0.1)
    else:
        r, adapters = case["rank"], case["adapters"]
        state["w"] = normal(n, k, scale=k ** -0.5)
        state["a"] = normal(adapters, r, k, scale=k ** -0.5)
        state["b"] = normal(adapters, n, r, scale=r ** -0.5)
        # about one request in eight has no adapter
        ids = np.where(rng.random(segments) < 0.125, -1, rng.integers(0, adapters, segments))
        state["adapter"] = torch.from_numpy(ids.astype(np.int32)).cuda()
        state["scale"] = torch.from_numpy(rng.uniform(0.25, 2.0, adapters).astype(np.float32)).cuda()
    return state


def _cut(case, offsets, rows):
    """The chunks of the plain form: (segment of each chunk, rows of each chunk [chunks, C], which of them are real)."""
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


def _run_plain(state):
    case, offsets, x = state["case"], state["offsets"], state["x"]
    seg, row, real = _cut(case, offsets, x.shape[0])
    xc = x[row].float() * real[..., None]
    if case["op"] == "gw":
        parts = torch.bmm(xc.transpose(1, 2), state["dy"][row].float())
        out = torch.zeros(case["segments"], case["k"], case["n"], device=x.device)
        out.index_add_(0, seg, parts)
        return out if case["out"] == "f32" else out.to(x.dtype)
    if case["op"] == "mm":
        wc = state["w"][seg].float()
        yc = torch.bmm(xc, wc.transpose(1, 2) if case["trans"] else wc)
        out = torch.zeros(x.shape[0], case["n"], device=x.device)
    else:
        ids = state["adapter"][seg].long()
        used = (ids >= 0)[:, None, None]
        ids = ids.clamp(min=0)
        uc = torch.bmm(xc, state["a"][ids].float().transpose(1, 2)) * state["scale"][ids][:, None, None]
        yc = torch.bmm(uc * used, state["b"][ids].float().transpose(1, 2))
        out = x.float() @ state["w"].float().t()
    # rows that pad a chunk add nothing to the row they were clamped to
    return out.index_add_(0, row.reshape(-1), (yc * real[..., None]).flatten(0, 1)).to(x.dtype)


def run(state):
    if not own:
        return _run_plain(state)
    import segmented_reduction_csr_gb300 as sr
    case, offsets = state["case"], state["offsets"]
    if case["op"] == "mm":
        return sr.seg_matmul(state["x"], state["w"], offsets, transpose_w=case["trans"])
    if case["op"] == "gw":
        return sr.seg_matmul_grad_w(state["x"], state["dy"], offsets,
                                    out_dtype=torch.float32 if case["out"] == "f32" else None)
    return sr.seg_lora(state["x"], state["w"], state["a"], state["b"], offsets, state["adapter"], state["scale"])


def work(case):
    rows, k, n, size = case["rows"], case["k"], case["n"], SIZE[case["dtype"]]
    total = rows + case["pad"]
    if case["op"] == "mm":
        # the rows of segments are read, every row of the output is written; at most `rows` matrices are needed
        b = size * (rows * k + min(rows, case["segments"]) * k * n + total * n) + 8 * (case["segments"] + 1)
        return {"bytes": b, "flops": 2.0 * rows * k * n}
    if case["op"] == "gw":
        osize = 4 if case["out"] == "f32" else size
        b = size * rows * (k + n) + osize * case["segments"] * k * n + 8 * (case["segments"] + 1)
        return {"bytes": b, "flops": 2.0 * rows * k * n}
    r = case["rank"]
    used = min(case["adapters"], case["segments"])
    b = size * (total * k + n * k + used * r * (k + n) + total * n) + 12 * (case["segments"] + 1)
    return {"bytes": b, "flops": 2.0 * total * k * n + 2.0 * rows * r * (k + n)}


def exact(case, seed):
    state = prepare(case, seed)
    x = state["x"].double()
    off = state["offsets"].tolist()
    pairs = [(s, slice(off[s], off[s + 1])) for s in range(case["segments"]) if off[s + 1] > off[s]]
    if case["op"] == "gw":
        out = x.new_zeros(case["segments"], case["k"], case["n"])
        for s, at in pairs:
            out[s] = x[at].t() @ state["dy"][at].double()
        return out
    if case["op"] == "mm":
        out = x.new_zeros(x.shape[0], case["n"])
        for s, at in pairs:
            w = state["w"][s].double()
            out[at] = x[at] @ (w.t() if case["trans"] else w)
        return out
    out = x @ state["w"].double().t()
    ids, scale = state["adapter"].tolist(), state["scale"].double().tolist()
    for s, at in pairs:
        i = ids[s]
        if i >= 0:
            out[at] += scale[i] * (x[at] @ state["a"][i].double().t()) @ state["b"][i].double().t()
    return out
