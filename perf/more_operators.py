"""The operators around the backward pass and the compressor: measured cases.

Three operators complete the training step whose gradient the compressor takes:

* ``embed`` -- the first layer: embedding lookup with a scale, and the table's gradient, which is written into (or
  added to) the flat gradient from the tokens sorted by their ids;
* ``rms``   -- root-mean-square norm behind the residual's addition.  The forward pass takes the layer's output and the
  residual stream, h = x + res, and gives h, y = norm(h) and an output in 8 bits with scales (the checkpoint that the
  weight gradient of the linear layer behind it reads), and keeps h in 8 bits or whole; the backward pass adds the
  gradient that comes along the residual stream;
* ``orth``  -- the last step: the update, orthogonalised by Newton-Schulz products before it is applied.

The 8-bit format of a [rows, cols] activation: groups of 32 consecutive columns share one scale byte B, the biased
binary32 exponent of the group's largest magnitude plus one; an element is one byte, sign << 7 | m with m = min(127,
round_half_even(|x| * 2^(134 - B))) and no sign when m = 0; it stands for +-m * 2^(B - 134).  B = 0: every element below
2^-120, all zero.  B = 255: a NaN, an infinity or a magnitude of 2^127 and more in the group, which restores as NaN.
Codes lie in rows of round_up(cols, 32) bytes, scale bytes in rows of round_up(ceil(cols / 32), 16).
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
STEPS, COEFS, ORTH_EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7  # the usual quintic and number of steps
PAD = -1  # the id of padding tokens


def listed():
    return [
        # one token of a batch of one looked up in a table of 32768 x 4096: latency is all
        {"name": "embed_one", "op": "embed", "tokens": 1, "vocab": 32768, "cols": 4096, "pad": 0, "dtype": "bf16", "ids": "i64", "grad": False, "accumulate": False},
        # a short batch through a small table, with its gradient
        {"name": "embed_small", "op": "embed", "tokens": 100, "vocab": 1000, "cols": 512, "pad": 0, "dtype": "bf16", "ids": "i64", "grad": True, "accumulate": False},
        # 16384 tokens of a training step: the gradient of the whole table is written, most of its rows as zeros
        {"name": "embed_train", "op": "embed", "tokens": 16384, "vocab": 32768, "cols": 4096, "pad": 0, "dtype": "bf16", "ids": "i64", "grad": True, "accumulate": False},
        # a further micro-batch: the gradient is added to the rows that occur; fp32, odd sizes, rows inside a wider buffer
        {"name": "embed_ragged_f32", "op": "embed", "tokens": 5003, "vocab": 50021, "cols": 1001, "pad": 2, "dtype": "f32", "ids": "i32", "grad": True, "accumulate": True},
        # one token through the norm of a 4096-wide layer, forward only
        {"name": "rms_one_row", "op": "rms", "rows": 1, "cols": 4096, "pad": 0, "dtype": "bf16", "ckpt": False, "whole": True, "grad": False},
        # the norm over 16384 tokens of a training step: h in 8 bits for the backward pass, y whole and in 8 bits
        {"name": "rms_train", "op": "rms", "rows": 16384, "cols": 4096, "pad": 0, "dtype": "bf16", "ckpt": True, "whole": True, "grad": True},
        # fp32 training, an odd width, rows inside a wider buffer, h kept whole
        {"name": "rms_ragged_f32", "op": "rms", "rows": 3001, "cols": 4099, "pad": 2, "dtype": "f32", "ckpt": False, "whole": True, "grad": True},
        # fp16, the width of a gated hidden layer, y in 8 bits alone
        {"name": "rms_wide_f16", "op": "rms", "rows": 2048, "cols": 11008, "pad": 0, "dtype": "f16", "ckpt": True, "whole": False, "grad": True},
        # the update of a small layer
        {"name": "orth_small", "op": "orth", "m": 128, "n": 64, "pad": 0, "dtype": "f32"},
        # fp32, odd sizes, rows inside a wider buffer
        {"name": "orth_ragged_f32", "op": "orth", "m": 1001, "n": 2051, "pad": 2, "dtype": "f32"},
        # the square projection of a 4096-wide layer, from the flat fp32 gradient
        {"name": "orth_square_f32", "op": "orth", "m": 4096, "n": 4096, "pad": 0, "dtype": "f32"},
        # the up projection 4096 -> 11008, a bf16 momentum: the largest update of the layer
        {"name": "orth_tall_bf16", "op": "orth", "m": 11008, "n": 4096, "pad": 0, "dtype": "bf16"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm; about half of them multiples of 64."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if n >= 64 and rng.random() < 0.5:
        n = n // 64 * 64
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(["embed", "rms", "orth"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16", "f32", "f32"]), "pad": rng.choice([0, 0, 0, 3, 32])}
    if op == "embed":
        case["ids"], case["grad"] = rng.choice(["i32", "i64"]), rng.random() < 0.8
        case["accumulate"] = case["grad"] and rng.random() < 0.4
        while True:
            case["tokens"], case["vocab"], case["cols"] = _spread(rng, 1, 32768), _spread(rng, 64, 65536), _spread(rng, 33, 8192)
            if case["tokens"] * case["cols"] <= 16384 * 4096 and case["vocab"] * case["cols"] <= 32768 * 4096:
                return case
    if op == "rms":
        case["ckpt"], case["whole"], case["grad"] = rng.random() < 0.6, rng.random() < 0.7, rng.random() < 0.8
        while True:
            case["rows"], case["cols"] = _spread(rng, 1, 32768), _spread(rng, 33, 16384)
            if case["rows"] * case["cols"] <= 16384 * 4096:
                return case
    while True:
        case["m"], case["n"] = _spread(rng, 17, 11008), _spread(rng, 17, 11008)
        if case["m"] * case["n"] * min(case["m"], case["n"]) <= 4096 * 4096 * 11008:
            return case


# --- the 8-bit format in elementary operations ----------------------------------------------------

def pitches(cols):
    """Bytes of one row of codes and of one row of scale bytes."""
    codes = -(-cols // 32) * 32
    return codes, -(-(codes // 32) // 16) * 16


def encode(x):
    """Codes and scale bytes of x (binary32, [rows, cols])."""
    rows, cols = x.shape
    pc, ps = pitches(cols)
    g = torch.nn.functional.pad(x, (0, pc - cols)).view(rows, pc // 32, 32)
    field = (g.abs().amax(2).view(torch.int32) >> 23) & 0xFF
    field = torch.where(g.isnan().any(2), 255, field)
    b = torch.where(field < 7, 0, torch.where(field >= 254, 255, field + 1)).to(torch.int32)
    real = (b > 0) & (b < 255)
    up = torch.where(real, (261 - b) << 23, 0).to(torch.int32).view(torch.float32)
    m = torch.where(real[..., None], (g.abs() * up[..., None]).round().clamp(max=127), 0.0)
    code = m.to(torch.int32) + torch.where((g < 0) & (m > 0), 128, 0)
    scales = torch.zeros(rows, ps, dtype=torch.uint8, device=x.device)
    scales[:, :pc // 32] = b.to(torch.uint8)
    return code.to(torch.uint8).view(rows, pc), scales


def decode(codes, scales, cols):
    """The binary32 values that codes and scale bytes stand for."""
    rows, pc = codes.shape
    b = scales[:, :pc // 32].to(torch.int32)
    s = torch.where((b > 7) & (b < 255), (b - 7) << 23, 0).to(torch.int32).view(torch.float32)
    s = torch.where(b == 255, math.nan, s)
    c = codes.view(rows, pc // 32, 32).to(torch.int32)
    v = (c & 127).to(torch.float32) * s[..., None]
    v = torch.where(c > 127, -v, v)
    return v.view(rows, pc)[:, :cols]


# --- inputs --------------------------------------------------------------------------------------

def _buffer(rows, cols, pad, dtype):
    return torch.zeros(rows, cols + pad, dtype=dtype, device="cuda")[:, :cols]


def _activation(gen, rows, cols, pad, dtype, size=1.0):
    """Activations: a scale for each column, a few columns far above the others, a few empty (padding) rows."""
    dev = "cuda"
    col = size * torch.exp(0.5 * torch.randn(cols, generator=gen, device=dev))
    col = torch.where(torch.rand(cols, generator=gen, device=dev) < 0.003, 20.0 * col, col)
    x = _buffer(rows, cols, pad, dtype)
    keep = torch.rand(rows, 1, generator=gen, device=dev) >= 0.01
    x.copy_(torch.randn(rows, cols, generator=gen, device=dev).mul_(col).mul_(keep))
    return x


def _gradient(gen, rows, cols, pad, dtype):
    """An output's gradient: small, a size for each row (fp16 comes scaled up by the loss scale)."""
    dev = "cuda"
    row = torch.exp(torch.randn(rows, 1, generator=gen, device=dev)) * (1.0 if dtype == torch.float16 else 1e-3)
    d = _buffer(rows, cols, pad, dtype)
    d.copy_(torch.randn(rows, cols, generator=gen, device=dev).mul_(row))
    return d


def _tokens(gen, tokens, vocab, itype):
    """Ids by frequency as of words (the v-th most frequent one's share falls as 1 / (v + 3)), spread over the table,
    with 1 % of padding."""
    dev = "cuda"
    share = torch.cumsum(1.0 / (torch.arange(vocab, dtype=torch.float64, device=dev) + 3.0), 0)
    at = torch.searchsorted(share, torch.rand(tokens, generator=gen, device=dev, dtype=torch.float64) * share[-1])
    ids = torch.randperm(vocab, generator=gen, device=dev)[at.clamp(max=vocab - 1)]
    ids = torch.where(torch.rand(tokens, generator=gen, device=dev) < 0.01, PAD, ids)
    return ids.to(torch.int32 if itype == "i32" else torch.int64)


def _update(gen, m, n, pad, dtype):
    """A momentum: a few strong directions above noise, a size for each row."""
    dev = "cuda"
    r = max(1, min(m, n) // 16)
    fall = torch.exp(-4.0 * torch.arange(r, device=dev) / r)
    low = (torch.randn(m, r, generator=gen, device=dev) * fall) @ torch.randn(r, n, generator=gen, device=dev) / math.sqrt(r)
    g = _buffer(m, n, pad, dtype)
    row = 1e-3 * torch.exp(0.3 * torch.randn(m, 1, generator=gen, device=dev))
    g.copy_(low.add_(torch.randn(m, n, generator=gen, device=dev)).mul_(row))
    return g


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    pad, dtype = case["pad"], DTYPES[case["dtype"]]
    f32 = {"dtype": torch.float32, "device": "cuda"}
    u8 = {"dtype": torch.uint8, "device": "cuda"}
    s = {"case": case}
    if case["op"] == "embed":
        tokens, vocab, cols = case["tokens"], case["vocab"], case["cols"]
        s["ids"] = _tokens(gen, tokens, vocab, case["ids"])
        s["table"] = _buffer(vocab, cols, pad, dtype)
        s["table"].copy_(torch.randn(vocab, cols, generator=gen, device="cuda").mul_(0.02))
        s["scale"] = math.sqrt(cols)
        s["y"] = _buffer(tokens, cols, pad, dtype)
        if case["grad"]:
            s["dy"] = _gradient(gen, tokens, cols, pad, dtype)
            s["dtable"] = torch.empty(vocab, cols, **f32)
            if case["accumulate"]:
                s["dtable"].copy_(torch.randn(vocab, cols, generator=gen, device="cuda").mul_(1e-3))
        return s
    if case["op"] == "rms":
        rows, cols = case["rows"], case["cols"]
        pc, ps = pitches(cols)
        s["x"] = _activation(gen, rows, cols, pad, dtype, 0.3)
        s["res"] = _activation(gen, rows, cols, pad, dtype)
        s["gamma"] = 1.0 + 0.1 * torch.randn(cols, generator=gen, **f32)
        s["h"] = _buffer(rows, cols, pad, dtype)
        s["y"] = _buffer(rows, cols, pad, dtype) if case["whole"] else None
        s["rstd"] = torch.empty(rows, **f32)
        s["y_codes"], s["y_scales"] = torch.empty(rows, pc, **u8), torch.empty(rows, ps, **u8)
        s["y8"] = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")  # the 8 bits restored: exact in bf16
        s["codes"], s["scales"] = (torch.empty(rows, pc, **u8), torch.empty(rows, ps, **u8)) if case["ckpt"] else (None, None)
        if case["grad"]:
            s["dy"], s["dres"] = _gradient(gen, rows, cols, pad, dtype), _gradient(gen, rows, cols, pad, dtype)
            s["dx"], s["dgamma"] = _buffer(rows, cols, pad, dtype), torch.empty(cols, **f32)
        return s
    s["g"] = _update(gen, case["m"], case["n"], pad, dtype)
    s["out"] = _buffer(case["m"], case["n"], pad, dtype)
    return s


# --- one pass ------------------------------------------------------------------------------------

_handle = None


def _context(scratch):
    """The program's one context, with room for `scratch` bytes."""
    global _handle
    from gradient_compression_ef_gb300 import gc
    if _handle is None:
        _handle = gc.Context(0)
    _handle.reserve_scratch(scratch)
    return _handle


def _run_own(s):
    from gradient_compression_ef_gb300 import gc
    case = s["case"]
    if case["op"] == "embed":
        tokens, vocab, cols = case["tokens"], case["vocab"], case["cols"]
        ctx = _context(gc.embedding_scratch_bytes(tokens, vocab, cols) if case["grad"] else 0)
        gc.embedding_forward(ctx, s["ids"], s["table"], s["scale"], s["y"], pad=PAD)
        if not case["grad"]:
            return {"y": s["y"]}
        gc.embedding_wgrad(ctx, s["dy"], s["ids"], s["scale"], s["dtable"], pad=PAD, accumulate=case["accumulate"])
        return {"y": s["y"], "dtable": s["dtable"]}
    if case["op"] == "rms":
        rows, cols = case["rows"], case["cols"]
        ctx = _context(gc.rmsnorm_scratch_bytes(rows, cols) if case["grad"] else 0)
        gc.rmsnorm_forward(ctx, s["x"], s["res"], s["gamma"], EPS, s["h"], s["y"], s["rstd"], s["codes"], s["scales"], s["y_codes"], s["y_scales"])
        gc.ckpt_restore(ctx, s["y_codes"], s["y_scales"], s["y8"])
        out = {"h": s["h"], "rstd": s["rstd"], "y8": s["y8"]}
        if case["whole"]:
            out["y"] = s["y"]
        if case["grad"]:
            gc.rmsnorm_backward(ctx, s["dy"], s["dres"], None if case["ckpt"] else s["h"], s["gamma"], s["rstd"], s["dx"], s["dgamma"], s["codes"], s["scales"])
            out["dx"], out["dgamma"] = s["dx"], s["dgamma"]
        return out
    ctx = _context(gc.orthogonalize_scratch_bytes(case["m"], case["n"]))
    gc.orthogonalize(ctx, s["g"], s["out"], steps=STEPS, coefs=COEFS, eps=ORTH_EPS, scale=math.sqrt(max(1.0, case["m"] / case["n"])))
    return {"out": s["out"]}


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "embed":
        ids = s["ids"].long()
        some = (ids != PAD)[:, None]
        y = (s["table"][ids.clamp(min=0)].float() * s["scale"] * some).to(dtype)
        if not case["grad"]:
            return {"y": y}
        d = s["dtable"] if case["accumulate"] else torch.zeros_like(s["dtable"])
        d.index_add_(0, ids.clamp(min=0), s["dy"].float() * s["scale"] * some)
        return {"y": y, "dtable": d}
    if case["op"] == "rms":
        cols, gamma = case["cols"], s["gamma"]
        h = (s["x"].float() + s["res"].float()).to(dtype)
        f = h.float()
        rstd = torch.rsqrt(f.square().mean(1, keepdim=True) + EPS)
        y = (f * rstd * gamma).to(dtype)
        out = {"h": h, "rstd": rstd[:, 0], "y8": decode(*encode(y.float()), cols).to(torch.bfloat16)}
        if case["whole"]:
            out["y"] = y
        if case["grad"]:
            dy = s["dy"].float()
            n = (decode(*encode(f), cols) if case["ckpt"] else f) * rstd
            d = dy * gamma
            out["dx"] = (rstd * (d - n * (d * n).mean(1, keepdim=True)) + s["dres"].float()).to(dtype)
            out["dgamma"] = (dy * n).sum(0)
        return out
    a, b, c = COEFS
    x = s["g"].float()
    x = x / (x.square().sum().sqrt() + ORTH_EPS)
    if case["m"] > case["n"]:
        x = x.t()
    for _ in range(STEPS):
        gram = x @ x.t()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    if case["m"] > case["n"]:
        x = x.t()
    return {"out": (x * math.sqrt(max(1.0, case["m"] / case["n"]))).to(dtype)}


def _distinct(tokens, vocab):
    """How many ids of _tokens' distribution occur in so many tokens, on average."""
    p = 1.0 / (torch.arange(vocab, dtype=torch.float64) + 3.0)
    return float((1.0 - torch.exp(0.99 * tokens * torch.log1p(-p / p.sum()))).sum())


def work(case):
    """What the calls of one pass need: the forward and the backward call of a step lie far apart, so what the
    backward call takes from the forward one is written and read."""
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "embed":
        tokens, cols, ids = case["tokens"], case["cols"], (4 if case["ids"] == "i32" else 8) * case["tokens"]
        rows = max(1.0, _distinct(tokens, case["vocab"]))
        need = {"bytes": ids + (rows + tokens) * cols * e, "flops": tokens * cols}
        if case["grad"]:  # the rows that occur are read and written, or the whole table is written
            need["bytes"] += ids + tokens * cols * e + 4 * cols * (2 * rows if case["accumulate"] else case["vocab"])
            need["flops"] += 2 * tokens * cols
        return need
    if op == "rms":  # x, res -> h, y, y in 8 bits (and h in 8 bits); the 8 bits -> their values; dy, dres, h -> dx
        rows, cols = case["rows"], case["cols"]
        n = rows * cols
        ckpt = n + n // 32
        nbytes = 3 * n * e + case["whole"] * n * e + 2 * ckpt + 2 * n + 4 * rows + 4 * cols
        if case["grad"]:
            nbytes += 3 * n * e + (2 * ckpt if case["ckpt"] else n * e) + 4 * rows + 8 * cols
        return {"bytes": nbytes, "flops": (20 if case["grad"] else 8) * n}
    m, n = case["m"], case["n"]
    small = min(m, n)
    # three products a step; the two that give symmetric matrices need half of theirs
    return {"bytes": 2 * m * n * e, "flops": STEPS * (3 * small * m * n + small ** 3)}


# --- the definitions in 64 bits ------------------------------------------------------------------

def _stands_for(x):
    """What the 8 bits of x (binary64, finite, below 2^127) stand for: the group's step is 2^(e - 7) with
    2^(e - 1) <= largest magnitude < 2^e; multiples of the step, at most 127 of them."""
    rows, cols = x.shape
    groups = -(-cols // 32)
    g = torch.zeros(rows, groups * 32, dtype=torch.float64, device=x.device)
    g[:, :cols] = x
    g = g.view(rows, groups, 32)
    top = g.abs().max(dim=2, keepdim=True).values
    step = torch.exp2(torch.frexp(top).exponent.to(torch.float64) - 7.0)
    got = torch.clamp(torch.round(g / step), -127.0, 127.0) * step
    got = torch.where(top < 2.0 ** -120, torch.zeros_like(got), got)
    return got.view(rows, groups * 32)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "embed":
        kept = torch.nonzero(s["ids"] != PAD)[:, 0]
        ids = s["ids"][kept].long()
        y = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        y[kept] = s["table"].index_select(0, ids).double() * s["scale"]
        if not case["grad"]:
            return {"y": y}
        d = s["dtable"].double() if case["accumulate"] else torch.zeros(case["vocab"], case["cols"], dtype=torch.float64, device="cuda")
        d.index_put_((ids,), s["dy"][kept].double() * s["scale"], accumulate=True)
        return {"y": y, "dtable": d}
    if case["op"] == "rms":
        cols, gamma = case["cols"], s["gamma"].double()
        h = s["x"].double() + s["res"].double()
        stored = (s["x"].float() + s["res"].float()).to(dtype).double()  # the norm is that of h as it is stored
        rstd = (torch.einsum("rc,rc->r", stored, stored) / cols + EPS) ** -0.5
        y = torch.einsum("rc,r,c->rc", stored, rstd, gamma)
        out = {"h": h, "rstd": rstd, "y8": _stands_for(y.to(dtype).double())}
        if case["whole"]:
            out["y"] = y
        if case["grad"]:
            dy = s["dy"].double()
            k = _stands_for(stored) if case["ckpt"] else stored
            dot = torch.einsum("rc,c,rc->r", dy, gamma, k)
            out["dx"] = torch.einsum("rc,c,r->rc", dy, gamma, rstd) - k * (rstd ** 3 * dot / cols)[:, None] + s["dres"].double()
            out["dgamma"] = torch.einsum("rc,rc,r->c", dy, k, rstd)
        return out
    # the polynomial of each step on the eigenvalues' side: p(X X^T) X with p in Horner's form
    a, b, c = COEFS
    x = s["g"].double()
    x = x / (torch.linalg.vector_norm(x) + ORTH_EPS)
    tall = case["m"] > case["n"]
    for _ in range(STEPS):
        gram = x.mT @ x if tall else x @ x.mT
        q = c * gram
        q.diagonal().add_(b)
        q = q @ gram
        q.diagonal().add_(a)
        x = x @ q if tall else q @ x
    return {"out": x * math.sqrt(max(1.0, case["m"] / case["n"]))}
