"""The operators of the backward pass that fills the flat gradient: measured cases.

Four operators stand before the compressor in a training step.  They produce,
from activations kept in 8 bits, the weight gradients that the compressor
takes:

* ``ckpt``   -- an activation saved in 8 bits and restored (the recompute path);
* ``act``    -- GELU / SiLU (optionally gated) forward, its input kept in 8 bits,
  and the backward pass from that checkpoint;
* ``norm``   -- layer norm forward (input kept in 8 bits, or whole) and backward,
  with the reduction of the weight's and bias's gradients over the rows;
* ``linear`` -- the weight and bias gradients of a linear layer from dy and the
  8-bit checkpoint of its input.

The checkpoint format (the same for every operator), for a [rows, cols] activation:
groups of 32 consecutive columns share one scale byte B, the biased binary32
exponent of the group's largest magnitude plus one; an element is one byte,
sign << 7 | m with m = min(127, round_half_even(|x| * 2^(134 - B))) and no sign
when m = 0; it stands for +-m * 2^(B - 134).  B = 0: every element below 2^-120,
all zero.  B = 255: a NaN, an infinity or a magnitude of 2^127 and more in the
group, which restores as NaN.  Codes lie in rows of round_up(cols, 32) bytes,
scale bytes in rows of round_up(ceil(cols / 32), 16).
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one token through a norm of a 4096-wide layer: a batch of one, where the calls' latency is all
        {"name": "norm_one_row", "op": "norm", "rows": 1, "cols": 4096, "pad": 0, "dtype": "bf16", "ckpt": True},
        # the norm of a 4096-wide layer over 16384 tokens of a training step
        {"name": "norm_train", "op": "norm", "rows": 16384, "cols": 4096, "pad": 0, "dtype": "bf16", "ckpt": True},
        # fp32 training, an odd width, rows inside a wider buffer, the input kept whole
        {"name": "norm_ragged_f32", "op": "norm", "rows": 3001, "cols": 4099, "pad": 2, "dtype": "f32", "ckpt": False},
        # GELU on a short ragged batch
        {"name": "act_small", "op": "act", "kind": "gelu", "gated": False, "rows": 17, "cols": 4096, "pad": 0, "dtype": "bf16"},
        # the gated hidden layer (11008 wide) of a training step
        {"name": "act_gated_train", "op": "act", "kind": "silu", "gated": True, "rows": 8192, "cols": 11008, "pad": 0, "dtype": "bf16"},
        # fp16, an odd width: rows that start on any even byte
        {"name": "act_ragged_f16", "op": "act", "kind": "gelu", "gated": False, "rows": 4093, "cols": 4097, "pad": 0, "dtype": "f16"},
        # save and restore of an fp32 activation
        {"name": "ckpt_f32", "op": "ckpt", "rows": 8192, "cols": 4096, "pad": 0, "dtype": "f32"},
        # save and restore, odd sizes, a small call
        {"name": "ckpt_ragged", "op": "ckpt", "rows": 333, "cols": 1001, "pad": 0, "dtype": "bf16"},
        # a small layer on a short batch
        {"name": "linear_small", "op": "linear", "rows": 100, "cols": 512, "out": 512, "pad": 0, "dtype": "bf16"},
        # the up projection 4096 -> 11008 over 8192 tokens: the largest weight gradient of the layer
        {"name": "linear_train", "op": "linear", "rows": 8192, "cols": 4096, "out": 11008, "pad": 0, "dtype": "bf16"},
        # fp32 dy, odd sizes in every direction, dy inside a wider buffer
        {"name": "linear_ragged_f32", "op": "linear", "rows": 2501, "cols": 1001, "out": 2051, "pad": 2, "dtype": "f32"},
        # a narrow layer over many tokens (the sum is long, the result small), fp16 dy
        {"name": "linear_long_f16", "op": "linear", "rows": 32768, "cols": 768, "out": 512, "pad": 0, "dtype": "f16"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm; about half of them multiples of 64."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if n >= 64 and rng.random() < 0.5:
        n = n // 64 * 64
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(["norm", "norm", "act", "act", "ckpt", "linear", "linear"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "pad": rng.choice([0, 0, 0, 3, 32])}
    while True:
        case["rows"] = _spread(rng, 1, 32768)
        case["cols"] = _spread(rng, 33, 16384)
        if op == "linear":
            case["out"] = _spread(rng, 33, 11008)
            planes = {"bf16": 1, "f16": 2, "f32": 3}[case["dtype"]]
            if planes * case["rows"] * case["cols"] * case["out"] <= 8192 * 4096 * 11008:
                break
        elif case["rows"] * case["cols"] <= 16384 * 4096:
            break
    if op == "act":
        case["kind"], case["gated"] = rng.choice(["gelu", "silu"]), rng.random() < 0.5
    if op == "norm":
        case["ckpt"] = rng.random() < 0.7
    return case


# --- the checkpoint format in elementary operations ---------------------------------------------

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

def _activation(gen, rows, cols, pad, dtype):
    """Activations: a scale for each column, a few columns far above the others, a few empty (padding) rows."""
    dev = "cuda"
    col = torch.exp(0.5 * torch.randn(cols, generator=gen, device=dev))
    col = torch.where(torch.rand(cols, generator=gen, device=dev) < 0.003, 20.0 * col, col)
    off = 0.3 * torch.randn(cols, generator=gen, device=dev)
    buf = torch.zeros(rows, cols + pad, dtype=dtype, device=dev)
    x = buf[:, :cols]
    v = torch.randn(rows, cols, generator=gen, device=dev).mul_(col).add_(off)
    keep = torch.rand(rows, 1, generator=gen, device=dev) >= 0.01
    x.copy_(v.mul_(keep))
    return x, keep


def _gradient(gen, rows, cols, pad, dtype, keep):
    """An output's gradient: small, a size for each row, zero at the empty rows (fp16 comes scaled up by the loss scale)."""
    dev = "cuda"
    row = torch.exp(torch.randn(rows, 1, generator=gen, device=dev)) * (1.0 if dtype == torch.float16 else 1e-3)
    buf = torch.zeros(rows, cols + pad, dtype=dtype, device=dev)
    d = buf[:, :cols]
    d.copy_(torch.randn(rows, cols, generator=gen, device=dev).mul_(row).mul_(keep))
    return d


def _ckpt_buffers(rows, cols):
    pc, ps = pitches(cols)
    return (torch.empty(rows, pc, dtype=torch.uint8, device="cuda"),
            torch.empty(rows, ps, dtype=torch.uint8, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rows, cols, pad, dtype = case["rows"], case["cols"], case["pad"], DTYPES[case["dtype"]]
    f32 = {"dtype": torch.float32, "device": "cuda"}
    s = {"case": case}
    x, keep = _activation(gen, rows, cols, pad, dtype)
    if case["op"] == "linear":
        s["codes"], s["scales"] = encode(x.float())
        s["dy"] = _gradient(gen, rows, case["out"], pad, dtype, keep)
        s["dw"], s["db"] = torch.empty(case["out"], cols, **f32), torch.empty(case["out"], **f32)
        return s
    s["x"], s["y"] = x, torch.empty(rows, cols, dtype=dtype, device="cuda")
    s["codes"], s["scales"] = _ckpt_buffers(rows, cols)
    if case["op"] == "ckpt":
        return s
    s["dy"], s["dx"] = _gradient(gen, rows, cols, pad, dtype, keep), torch.empty(rows, cols, dtype=dtype, device="cuda")
    if case["op"] == "act" and case["gated"]:
        s["gate"], _ = _activation(gen, rows, cols, pad, dtype)
        s["dgate"] = torch.empty(rows, cols, dtype=dtype, device="cuda")
        s["gate_codes"], s["gate_scales"] = _ckpt_buffers(rows, cols)
    if case["op"] == "norm":
        s["gamma"] = 1.0 + 0.1 * torch.randn(cols, generator=gen, **f32)
        s["beta"] = 0.1 * torch.randn(cols, generator=gen, **f32)
        s["mean"], s["rstd"] = torch.empty(rows, **f32), torch.empty(rows, **f32)
        s["dgamma"], s["dbeta"] = torch.empty(cols, **f32), torch.empty(cols, **f32)
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
    op, rows, cols = case["op"], case["rows"], case["cols"]
    if op == "ckpt":
        ctx = _context(0)
        gc.ckpt_save(ctx, s["x"], s["codes"], s["scales"])
        gc.ckpt_restore(ctx, s["codes"], s["scales"], s["y"])
        return {"x": s["y"]}
    if op == "act":
        ctx = _context(0)
        if case["gated"]:
            gc.act_forward(ctx, case["kind"], s["x"], s["y"], s["codes"], s["scales"], s["gate"], s["gate_codes"], s["gate_scales"])
            gc.act_backward(ctx, case["kind"], s["dy"], s["dx"], s["codes"], s["scales"], s["dgate"], s["gate_codes"], s["gate_scales"])
            return {"y": s["y"], "dx": s["dx"], "dgate": s["dgate"]}
        gc.act_forward(ctx, case["kind"], s["x"], s["y"], s["codes"], s["scales"])
        gc.act_backward(ctx, case["kind"], s["dy"], s["dx"], s["codes"], s["scales"])
        return {"y": s["y"], "dx": s["dx"]}
    if op == "norm":
        ctx = _context(gc.layernorm_scratch_bytes(rows, cols))
        if case["ckpt"]:
            gc.layernorm_forward(ctx, s["x"], s["gamma"], s["beta"], EPS, s["y"], s["mean"], s["rstd"], s["codes"], s["scales"])
            gc.layernorm_backward(ctx, s["dy"], None, s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"], s["codes"], s["scales"])
        else:
            gc.layernorm_forward(ctx, s["x"], s["gamma"], s["beta"], EPS, s["y"], s["mean"], s["rstd"])
            gc.layernorm_backward(ctx, s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"])
        return {k: s[k] for k in ("y", "mean", "rstd", "dx", "dgamma", "dbeta")}
    ctx = _context(gc.linear_wgrad_scratch_bytes(rows, case["out"], cols, case["dtype"]))
    gc.linear_wgrad(ctx, s["dy"], s["codes"], s["scales"], s["dw"], s["db"])
    return {"dw": s["dw"], "db": s["db"]}


def _act(kind, x):
    """f(x) and f'(x)."""
    if kind == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))
        return x * cdf, cdf + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
    sig = 1.0 / (1.0 + torch.exp(-x))
    return x * sig, sig * (1.0 + x * (1.0 - sig))


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    op, cols, dtype = case["op"], case["cols"], DTYPES[case["dtype"]]
    if op == "linear":
        x, dy = decode(s["codes"], s["scales"], cols), s["dy"].float()
        return {"dw": dy.t() @ x, "db": dy.sum(0)}
    x = s["x"].float()
    if op == "ckpt":
        return {"x": decode(*encode(x), cols).to(dtype)}
    dy = s["dy"].float()
    if op == "act":
        f, _ = _act(case["kind"], x)
        xs = decode(*encode(x), cols)
        fs, ds = _act(case["kind"], xs)
        if not case["gated"]:
            return {"y": f.to(dtype), "dx": (dy * ds).to(dtype)}
        gate = s["gate"].float()
        gs = decode(*encode(gate), cols)
        return {"y": (f * gate).to(dtype), "dx": (dy * gs * ds).to(dtype), "dgate": (dy * fs).to(dtype)}
    mean = x.mean(1, keepdim=True)
    rstd = torch.rsqrt((x - mean).square().mean(1, keepdim=True) + EPS)
    y = (x - mean) * rstd * s["gamma"] + s["beta"]
    xs = decode(*encode(x), cols) if case["ckpt"] else x
    n = (xs - mean) * rstd
    d = dy * s["gamma"]
    dx = rstd * (d - d.mean(1, keepdim=True) - n * (d * n).mean(1, keepdim=True))
    return {"y": y.to(dtype), "mean": mean[:, 0], "rstd": rstd[:, 0], "dx": dx.to(dtype),
            "dgamma": (dy * n).sum(0), "dbeta": dy.sum(0)}


def work(case):
    """What the calls of one pass need: the forward and the backward call of a step lie far apart, so what the
    backward call takes from the forward one (the checkpoint, the row statistics, or the whole input) is written and read."""
    op, rows, cols, e = case["op"], case["rows"], case["cols"], SIZE[case["dtype"]]
    n = rows * cols
    ckpt = n + n // 32
    if op == "ckpt":
        return {"bytes": 2 * n * e + 2 * ckpt, "flops": 4 * n}
    if op == "act":
        if case["gated"]:  # x, gate -> y, checkpoints; dy, checkpoints -> dx, dgate
            return {"bytes": 6 * n * e + 4 * ckpt, "flops": 40 * n}
        return {"bytes": 4 * n * e + 2 * ckpt, "flops": 30 * n}
    if op == "norm":  # x -> y (and the checkpoint); dy, x or checkpoint -> dx
        kept = 2 * ckpt if case["ckpt"] else n * e
        return {"bytes": 4 * n * e + kept + 16 * rows + 20 * cols, "flops": 22 * n}
    out = case["out"]
    return {"bytes": rows * out * e + ckpt + 4 * out * cols + 4 * out, "flops": 2 * rows * cols * out + rows * out}


# --- the definitions in 64 bits ------------------------------------------------------------------

def _stands_for(x):
    """What the checkpoint of x (binary64, finite, below 2^127) stands for: the group's step is 2^(e - 7) with
    2^(e - 1) <= largest magnitude < 2^e; multiples of the step, at most 127 of them."""
    rows, cols = x.shape
    groups = -(-cols // 32)
    g = torch.zeros(rows, groups * 32, dtype=torch.float64, device=x.device)
    g[:, :cols] = x
    g = g.view(rows, groups, 32)
    top = g.abs().max(dim=2, keepdim=True).values
    e = torch.frexp(top).exponent.to(torch.float64)
    step = torch.exp2(e - 7.0)
    got = torch.clamp(torch.round(g / step), -127.0, 127.0) * step
    got = torch.where(top < 2.0 ** -120, torch.zeros_like(got), got)
    return got.view(rows, groups * 32)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        # the value of code c at scale byte b, from a table over all bytes
        c = torch.arange(256, dtype=torch.float64, device="cuda")
        value = torch.where(c >= 128, 128.0 - c, c)
        x = value[s["codes"].long()]
        unit = torch.exp2(s["scales"].double() - 134.0)
        unit = torch.where(s["scales"] == 0, torch.zeros_like(unit), unit)
        x *= unit.repeat_interleave(32, dim=1)[:, :x.shape[1]]
        dy = s["dy"].double()
        return {"dw": torch.einsum("to,ti->oi", dy, x[:, :case["cols"]]), "db": dy.sum(dim=0)}
    x = s["x"].double()
    if op == "ckpt":
        return {"x": _stands_for(x)}
    dy = s["dy"].double()
    if op == "act":
        def f(v):
            if case["kind"] == "gelu":
                return v * torch.special.ndtr(v)
            return v * torch.sigmoid(v)

        def df(v):
            if case["kind"] == "gelu":
                return torch.special.ndtr(v) + v * torch.exp(-v * v / 2.0) / math.sqrt(2.0 * math.pi)
            p = torch.sigmoid(v)
            return p + v * p * torch.sigmoid(-v)

        xs = _stands_for(x)
        if not case["gated"]:
            return {"y": f(x), "dx": dy * df(xs)}
        gate = s["gate"].double()
        return {"y": f(x) * gate, "dx": dy * _stands_for(gate) * df(xs), "dgate": dy * f(xs)}
    var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
    rstd = 1.0 / torch.sqrt(var + EPS)
    gamma, beta = s["gamma"].double(), s["beta"].double()
    n = ((_stands_for(x) if case["ckpt"] else x) - mean) * rstd
    d, width = dy * gamma, x.shape[1]
    dx = (d - d.sum(1, keepdim=True) / width - n * ((d * n).sum(1, keepdim=True) / width)) * rstd
    return {"y": (x - mean) * rstd * gamma + beta, "mean": mean[:, 0], "rstd": rstd[:, 0], "dx": dx,
            "dgamma": (dy * n).sum(0), "dbeta": dy.sum(0)}
