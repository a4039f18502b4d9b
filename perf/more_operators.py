"""Measured cases of the final norm and of the 8-bit and 4-bit LM heads, with their plain forms.

Five operators that a server with speculative decoding runs next to the verify step:

  norm       RMS norm of hidden rows with the residual's addition, in the rows' type or as
             MXFP8 rows (blocks of 32 values, e4m3 codes, one power-of-two scale a block);
  quantise8  MXFP8 quantisation of rows, and the values the codes stand for;
  product8   logits of hidden rows under an MXFP8 LM head, the rows in MXFP8 already or
             quantised in the call;
  quantise4  4-bit integer weights with a scale (and a zero) per group of columns, and the
             values the codes stand for;
  product4   logits of unquantised hidden rows under such a 4-bit LM head.

`own` selects the side: False computes the plain forms (elementary torch operations), True
calls the library. `exact` states the same results in 64 bits, written apart.
"""
import functools
import math

import torch

own = False

BLOCK = 32                      # values that share one MXFP8 scale
TOP = 448.0                     # largest e4m3 magnitude
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the final norm of one request's next token: latency
        {"name": "norm-1", "op": "norm", "rows": 1, "d": 4096, "dtype": "bf16",
         "residual": "bf16", "weight": "bf16", "out": "same", "pad": 0},
        # the final norm of 128 requests' blocks of 17 rows, straight into the 8-bit LM head's form
        {"name": "norm-2176-mx", "op": "norm", "rows": 2176, "d": 7168, "dtype": "bf16",
         "residual": "bf16", "weight": "bf16", "out": "mx", "pad": 0},
        # one hidden row of each of 128 requests
        {"name": "quantise8-rows", "op": "quantise8", "rows": 128, "d": 4096, "dtype": "bf16"},
        # a whole LM head, once per model load
        {"name": "quantise8-head", "op": "quantise8", "rows": 129280, "d": 7168, "dtype": "bf16"},
        # one request's next drafted token, small head: the smallest call of a drafter
        {"name": "product8-1", "op": "product8", "rows": 1, "d": 2048, "V": 32768,
         "hidden": "bf16", "out": "bf16"},
        # the blocks of 16 of four requests, rows that the norm left in 8 bits
        {"name": "product8-64-mx", "op": "product8", "rows": 64, "d": 4096, "V": 151936,
         "hidden": "mx", "out": "fp32"},
        # a parallel drafter's blocks of 128 requests at once
        {"name": "product8-2048", "op": "product8", "rows": 2048, "d": 7168, "V": 129280,
         "hidden": "bf16", "out": "bf16"},
        # a small LM head, with zeros
        {"name": "quantise4-small", "op": "quantise4", "rows": 32768, "d": 2048, "dtype": "bf16",
         "group": 128, "symmetric": False},
        # a large one, fine groups without zeros
        {"name": "quantise4-head", "op": "quantise4", "rows": 151936, "d": 4096, "dtype": "fp16",
         "group": 32, "symmetric": True},
        # one request's next drafted token, small head
        {"name": "product4-1", "op": "product4", "rows": 1, "d": 2048, "V": 32768,
         "hidden": "bf16", "group": 128, "symmetric": False, "out": "bf16"},
        # one request's block of 16, fine groups
        {"name": "product4-16", "op": "product4", "rows": 16, "d": 4096, "V": 151936,
         "hidden": "fp16", "group": 32, "symmetric": True, "out": "fp32"},
        # four drafted rows of each of 128 requests
        {"name": "product4-512", "op": "product4", "rows": 512, "d": 7168, "V": 129280,
         "hidden": "bf16", "group": 128, "symmetric": False, "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quantise8", "product8", "quantise4", "product4"])
    kind = rng.choice(["bf16", "fp16", "fp32"])
    if op == "norm":
        out = rng.choice(["same", "mx"])
        d = _log_int(rng, 64, 16384)
        return {"op": op, "rows": _log_int(rng, 1, 16000), "d": d if out == "same" else d // 8 * 8,
                "dtype": kind, "residual": rng.choice(["none", kind, "fp32"]),
                "weight": rng.choice(["none", kind, "fp32"]), "out": out,
                "pad": rng.choice([0, 0, rng.randint(1, 100)])}
    if op == "quantise8":
        return {"op": op, "rows": _log_int(rng, 1, 100000), "d": 8 * _log_int(rng, 8, 896),
                "dtype": kind}
    out = rng.choice(["bf16", "fp32"])
    if op == "product8":
        return {"op": op, "rows": _log_int(rng, 1, 1500), "d": 8 * _log_int(rng, 16, 896),
                "V": _log_int(rng, 1000, 129000), "hidden": rng.choice(["mx", kind]), "out": out}
    group = rng.choice([32, 64, 128])
    d = group * _log_int(rng, 128 // group, 7168 // group)
    form = {"group": group, "symmetric": rng.random() < 0.5}
    if op == "quantise4":
        return {"op": op, "rows": _log_int(rng, 1, 100000), "d": d, "dtype": kind, **form}
    return {"op": op, "rows": _log_int(rng, 1, 500), "d": d, "V": _log_int(rng, 1000, 129000),
            "hidden": rng.choice(["bf16", "fp16"]), **form, "out": out}


_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "mx": 1 + 1 / BLOCK, "none": 0}


def _packed4(case):
    """Bytes a weight of the 4-bit form, scales and zeros counted in."""
    return 0.5 + (2 if case["symmetric"] else 3) / case["group"]


def work(case):
    op, rows, d = case["op"], case["rows"], case["d"]
    n = rows * d
    if op == "norm":
        res = _SIZE[case["residual"]]
        y = _SIZE[case["dtype"]] if case["out"] == "same" else 2 * _SIZE["mx"] + 2
        return {"bytes": n * (_SIZE[case["dtype"]] + 2 * res + y) + d * _SIZE[case["weight"]],
                "flops": 4 * n}
    if op == "quantise8":
        return {"bytes": n * (_SIZE[case["dtype"]] + 2 * _SIZE["mx"] + 2), "flops": 4 * n}
    if op == "quantise4":
        return {"bytes": n * (_SIZE[case["dtype"]] + 2 * _packed4(case) + 2), "flops": 6 * n}
    weights = _SIZE["mx"] if op == "product8" else _packed4(case)
    return {"bytes": n * _SIZE[case["hidden"]] + case["V"] * d * weights
            + rows * case["V"] * _SIZE[case["out"]], "flops": 2 * n * case["V"]}


# ------------------------------------------------------------------ inputs

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _hidden(rows, d, gen, kind):
    """Rows of a residual stream: unit columns, one in a hundred of them several times larger."""
    x = torch.randn((rows, d), generator=gen, device="cuda")
    big = torch.rand(d, generator=gen, device="cuda") < 0.01
    return x.mul_(torch.where(big, 12.0, 1.0)).to(_TYPES[kind])


def _weights(rows, d, gen, kind):
    """An LM head: rows of small values, some longer than others."""
    w = torch.randn((rows, d), generator=gen, device="cuda", dtype=_TYPES[kind])
    size = 0.01 + 0.02 * torch.rand((rows, 1), generator=gen, device="cuda")
    return w.mul_(size.to(w.dtype))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, rows, d = case["op"], case["rows"], case["d"]
    s = {"case": case}
    if op == "norm":
        s["x"] = _hidden(rows, d + case["pad"], gen, case["dtype"])[:, :d]
        s["residual"] = s["weight"] = None
        if case["residual"] != "none":
            s["residual"] = _hidden(rows, d, gen, case["residual"])
        if case["weight"] != "none":
            w = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda")
            s["weight"] = w.to(_TYPES[case["weight"]])
    elif op == "quantise8":
        s["x"] = _hidden(rows, d, gen, case["dtype"])
    elif op == "quantise4":
        s["x"] = _weights(rows, d, gen, case["dtype"])
    elif op == "product8":
        head = torch.nn.functional.pad(_weights(case["V"], d, gen, "bf16"), (0, -d % 128))
        s["codes"], s["scales"] = _mx_pack(*_mx_parts(head))
        if case["hidden"] == "mx":
            h = torch.nn.functional.pad(_hidden(rows, d, gen, "bf16"), (0, -d % 128))
            s["hidden"] = _mx_pack(*_mx_parts(h))
        else:
            s["hidden"] = _hidden(rows, d, gen, case["hidden"])
    else:
        s["hidden"] = _hidden(rows, d, gen, case["hidden"])
        code, scale, zero = _w4_parts(_weights(case["V"], d, gen, "bf16"), case["group"],
                                      case["symmetric"], torch.bfloat16)
        code = code.to(torch.uint8)
        s["codes"] = code[:, 0::2] | (code[:, 1::2] << 4)
        s["scales"] = scale
        s["zeros"] = None if case["symmetric"] else zero.to(torch.uint8)
    if own:
        _own_prepare(s)
    return s


def run(s):
    if own:
        return _own_run(s)
    return {"norm": _plain_norm, "quantise8": _plain_quantise8, "product8": _plain_product8,
            "quantise4": _plain_quantise4, "product4": _plain_product4}[s["case"]["op"]](s)


# ------------------------------------------------------------------ plain forms

@functools.lru_cache(maxsize=None)
def _powers(device):
    return torch.tensor([2.0 ** k for k in range(-149, 128)], device=device)


def _times_power(x, exponent):
    """x * 2^exponent; the powers from a table, as a power function may round."""
    return x * _powers(x.device)[exponent.long() + 149]


def _mx_parts(x):
    """e4m3 values (fp32, before the scale) [rows][d] and scale exponents (int32) of each
    block; a row's last block may be short."""
    rows, d = x.shape
    b = torch.nn.functional.pad(x.float(), (0, -d % BLOCK)).view(rows, -1, BLOCK)
    top = b.abs().amax(2)
    exponent = (torch.frexp(top)[1] - 9).clamp(-127, 127)      # floor(log2(top)) - 8
    exponent = torch.where(top > 0, exponent, torch.full_like(exponent, -127))
    y = _times_power(b, -exponent[:, :, None]).clamp(-TOP, TOP)
    # round to three bits behind the leading one, from 2^-6 down to steps of 2^-9 (ties to even)
    step = torch.frexp(y)[1].clamp(min=-5) - 4
    y = _times_power(torch.round(_times_power(y, -step)), step)
    return y.view(rows, -1)[:, :d], exponent.to(torch.int32)


def _mx_pack(value, exponent):
    """A byte a value; a scale is its exponent + 127."""
    return value.to(torch.float8_e4m3fn).view(torch.uint8), (exponent + 127).to(torch.uint8)


def _mx_values(value, exponent):
    rows, d = value.shape
    v = torch.nn.functional.pad(value, (0, -d % BLOCK)).view(rows, -1, BLOCK)
    return _times_power(v, exponent[:, :, None]).view(rows, -1)[:, :d]


def _mx_unpack(codes, scales):
    return _mx_values(codes.view(torch.float8_e4m3fn).float(), scales.to(torch.int32) - 127)


def _plain_norm(s):
    case, x, res, w = s["case"], s["x"], s["residual"], s["weight"]
    out = {}
    if res is not None:
        x = out["sum"] = (x.float() + res.float()).to(res.dtype)
    x = x.double() if case["out"] == "mx" else x.float()       # 8-bit codes have borders
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    if w is not None:
        y = y * w.to(y.dtype)
    if case["out"] == "mx":
        out["y"] = _mx_values(*_mx_parts(y.float())).to(torch.bfloat16)
    else:
        out["y"] = y.to(_TYPES[case["dtype"]])
    return out


def _plain_quantise8(s):
    return _mx_values(*_mx_parts(s["x"])).to(torch.bfloat16)     # every value is a bf16 number


def _plain_product8(s):
    d = s["case"]["d"]
    if s["case"]["hidden"] == "mx":
        h = _mx_unpack(*s["hidden"])[:, :d]
    else:
        h = _mx_values(*_mx_parts(s["hidden"]))
    w = _mx_unpack(s["codes"], s["scales"])[:, :d]
    return (h @ w.t()).to(_TYPES[s["case"]["out"]])


def _w4_parts(x, group, symmetric, kind):
    """Codes 0 .. 15 [rows][d] and, of each group, the scale (in `kind`) and the zero."""
    rows, d = x.shape
    b = x.float().view(rows, d // group, group)
    if symmetric:
        scale = (b.abs().amax(2) / 7).to(kind)
    else:
        hi, lo = b.amax(2).clamp(min=0), b.amin(2).clamp(max=0)
        scale = ((hi.double() - lo.double()) / 15).float().to(kind)
    f = scale.float()
    by = torch.where(f > 0, f, 1.0)[:, :, None]
    q = torch.where(f[:, :, None] > 0, torch.round(b / by), 0.0)
    if symmetric:
        zero = torch.full_like(f, 8)
    else:
        zero = torch.where(f > 0, torch.round(-lo / by[:, :, 0]).clamp(0, 15), 0.0)
    return (q + zero[:, :, None]).clamp(0, 15).view(rows, d), scale, zero


def _w4_values(code, scale, zero):
    rows, d = code.shape
    c = code.float().view(rows, scale.shape[1], -1)
    return ((c - zero.float()[:, :, None]) * scale.float()[:, :, None]).view(rows, d)


def _scale_type(s):
    return torch.bfloat16 if s["x"].dtype == torch.float32 else s["x"].dtype


def _plain_quantise4(s):
    c = s["case"]
    return _w4_values(*_w4_parts(s["x"], c["group"], c["symmetric"], _scale_type(s))).to(
        torch.bfloat16)


def _plain_product4(s):
    code = torch.stack([s["codes"] & 15, s["codes"] >> 4], 2).flatten(1)
    zero = torch.full_like(s["scales"], 8) if s["zeros"] is None else s["zeros"]
    w = _w4_values(code, s["scales"], zero)
    return (s["hidden"].float() @ w.t()).to(_TYPES[s["case"]["out"]])


# ------------------------------------------------------------------ the library's calls

def _own_prepare(s):
    import draft_block_verification_amd as sd
    case = s["case"]
    if case["op"] == "product8":
        # the LM head in the form that the product reads, made once per model load
        s["head"] = sd.Mxfp8Weights(s["codes"], s["scales"], case["d"])
        s["workspace"] = None
        if case["hidden"] != "mx":
            s["workspace"] = sd.new_workspace(
                sd.mxfp8_logits_workspace_bytes(case["rows"], case["d"]), s["codes"].device)
    elif case["op"] == "product4":
        s["head"] = sd.W4Weights(s["codes"], s["scales"], s["zeros"], case["d"])
        s["workspace"] = sd.new_workspace(
            sd.w4_logits_workspace_bytes(case["rows"], case["d"], case["group"]),
            s["codes"].device)


def _own_run(s):
    import draft_block_verification_amd as sd
    case = s["case"]
    op, d = case["op"], case["d"]
    if op == "norm":
        out, total = {}, None
        if s["residual"] is not None:
            total = out["sum"] = torch.empty_like(s["residual"])
        if case["out"] == "mx":
            codes, scales = sd.sd_rms_norm_mxfp8(s["x"], s["weight"], s["residual"], eps=EPS,
                                                 total=total)
            out["y"] = sd.sd_mxfp8_dequantize(codes, scales, d, dtype=torch.bfloat16)
        else:
            out["y"] = sd.sd_rms_norm(s["x"], s["weight"], s["residual"], eps=EPS, total=total)
        return out
    if op == "quantise8":
        return sd.sd_mxfp8_dequantize(*sd.sd_mxfp8_quantize(s["x"]), d, dtype=torch.bfloat16)
    if op == "quantise4":
        codes, scales, zeros = sd.sd_w4_quantize(s["x"], case["group"], case["symmetric"],
                                                 scale_dtype=_scale_type(s))
        return sd.sd_w4_dequantize(codes, scales, zeros, d, dtype=torch.bfloat16)
    product = sd.sd_mxfp8_logits if op == "product8" else sd.sd_w4_logits
    return product(s["hidden"], s["head"], dtype=_TYPES[case["out"]], workspace=s["workspace"])


# ------------------------------------------------------------------ in 64 bits

def _e4m3():
    """The magnitudes that e4m3 has, by code."""
    m = torch.arange(8, dtype=torch.float64)
    rows = [m * 2.0 ** -9] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16)]
    return torch.cat(rows)[:127].cuda()                 # the last code is NaN


def _exact_mx(x):
    """Values of the MXFP8 form of x (float64): nearest e4m3 number under the block's scale, by
    the distance to both neighbours (ties go to the even code)."""
    grid = _e4m3()
    scales = torch.tensor([2.0 ** e for e in range(-127, 128)], dtype=torch.float64, device="cuda")
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 24) // x.shape[1])
    for r in range(0, x.shape[0], step):
        b = torch.nn.functional.pad(x[r:r + step].double(), (0, -x.shape[1] % BLOCK))
        b = b.unflatten(1, (-1, BLOCK))
        top = b.abs().amax(2, keepdim=True)
        # the largest power of two whose 256-fold the block reaches
        scale = scales[(torch.bucketize(top / 256, scales, right=True) - 1).clamp(min=0)]
        a = (b.abs() / scale).clamp(max=TOP)
        lo = torch.bucketize(a, grid, right=True) - 1
        hi = (lo + 1).clamp(max=126)
        up, down = grid[hi] - a, a - grid[lo]
        code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        out[r:r + step] = (grid[code] * scale * torch.sign(b)).flatten(1)[:, :x.shape[1]]
    return out


def _exact_mx_bytes(codes, scales):
    c = codes.long()
    v = torch.cat([_e4m3(), torch.full((1,), math.nan, dtype=torch.float64, device="cuda")])
    w = v[c % 128] * (1.0 - 2.0 * (c // 128))
    power = torch.tensor([2.0 ** (k - 127) for k in range(256)], dtype=torch.float64, device="cuda")
    return w * power[scales.long()].repeat_interleave(BLOCK, 1)


def exact(case, seed):
    op, d = case["op"], case["d"]
    s = prepare(case, seed)
    if op == "norm":
        x, out = s["x"].double(), {}
        if s["residual"] is not None:
            out["sum"] = x + s["residual"].double()
            # the norm is that of the sum as it is kept
            x = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype).double()
        y = x / torch.sqrt(x.square().sum(1, keepdim=True) / d + EPS)
        y = y if s["weight"] is None else y * s["weight"].double()
        out["y"] = _exact_mx(y) if case["out"] == "mx" else y
        return out
    if op == "quantise8":
        return _exact_mx(s["x"])
    if op == "quantise4":
        x, g = s["x"], case["group"]
        out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
        step = max(1, (1 << 25) // d)
        for r in range(0, x.shape[0], step):
            b = x[r:r + step].double().unflatten(1, (-1, g))
            up, down = b.max(2, keepdim=True)[0], b.min(2, keepdim=True)[0]
            if case["symmetric"]:
                t = (torch.maximum(up, -down) / 7).float().to(_scale_type(s)).double()
                code = torch.round(b / t).clamp(-8, 7)
            else:
                up, down = up.clamp(min=0), down.clamp(max=0)
                t = ((up - down) / 15).float().to(_scale_type(s)).double()
                zero = torch.round(-down / t).clamp(0, 15)
                code = (torch.round(b / t) + zero).clamp(0, 15) - zero
            out[r:r + step] = torch.where(t > 0, code * t, 0.0).flatten(1)
        return out
    if op == "product8":
        h = _exact_mx_bytes(*s["hidden"])[:, :d] if case["hidden"] == "mx" else _exact_mx(s["hidden"])
    else:
        h = s["hidden"].double()
    out = torch.empty((case["rows"], case["V"]), dtype=torch.float64, device="cuda")
    for v in range(0, case["V"], 8192):
        if op == "product8":
            w = _exact_mx_bytes(s["codes"][v:v + 8192], s["scales"][v:v + 8192])[:, :d]
        else:
            c = s["codes"][v:v + 8192].double()
            high = torch.floor(c / 16)
            w = torch.stack([c - 16 * high, high], 2).flatten(1).unflatten(1, (-1, case["group"]))
            z = 8.0 if s["zeros"] is None else s["zeros"][v:v + 8192].double()[:, :, None]
            w = ((w - z) * s["scales"][v:v + 8192].double()[:, :, None]).flatten(1)
        out[:, v:v + 8192] = h @ w.t()
    return out
