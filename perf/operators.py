"""Measured cases of the drafter's and the sampler's operators, with their plain forms.

Four operators that a server with speculative decoding runs around the verify step:

  quantise  MXFP4 quantisation of bf16 rows (blocks of 32 values, e2m1 codes, one
            power-of-two scale per block) and the values the codes stand for;
  product   logits of hidden rows under an MXFP4 LM head, the hidden rows quantised in
            the call (the drafter's LM head: verification keeps the output lossless
            whatever the drafter's precision);
  sample    one token per row under temperature, top-k, top-p and min-p, by inverse CDF
            from a given uniform, with the size of the kept set and the log-probability;
  accept    rejection acceptance of a drafted block when target and drafter are both
            filtered that way: kept prefix, correction or bonus token.

`own` selects the side: False computes the plain forms (elementary torch operations), True
calls the library. `exact` states the same results in 64 bits, written apart.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 32                      # values that share one scale
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # e2m1 magnitudes by code


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one drafted token each of 128 requests: the hidden rows of a drafter step
        {"name": "quantise-rows", "op": "quantise", "rows": 128, "d": 4096, "dtype": "bf16"},
        # a whole LM head, once per model load
        {"name": "quantise-head", "op": "quantise", "rows": 129280, "d": 7168, "dtype": "bf16"},
        # one request's next drafted token, small head: the smallest call of a drafter
        {"name": "product-1", "op": "product", "rows": 1, "d": 2048, "V": 32768, "out": "bf16"},
        # a parallel drafter's whole block of one request
        {"name": "product-16", "op": "product", "rows": 16, "d": 4096, "V": 151936, "out": "fp32"},
        # one drafted token each of 128 requests
        {"name": "product-128", "op": "product", "rows": 128, "d": 7168, "V": 129280, "out": "bf16"},
        # a parallel drafter's blocks of 128 requests at once
        {"name": "product-2048", "op": "product", "rows": 2048, "d": 7168, "V": 129280, "out": "bf16"},
        # one request's token, common settings (latency)
        {"name": "sample-1", "op": "sample", "rows": 1, "V": 151936, "dtype": "fp32",
         "mix": "usual", "masked": False},
        # a batch of requests with settings of their own, a grammar's mask on every fourth row
        {"name": "sample-128-mixed", "op": "sample", "rows": 128, "V": 129280, "dtype": "bf16",
         "mix": "mixed", "masked": True},
        # every position of a large batch, top-p alone (the kept sets are long)
        {"name": "sample-1088-top-p", "op": "sample", "rows": 1088, "V": 151936, "dtype": "fp32",
         "mix": "top_p", "masked": False},
        # one request's block of 16
        {"name": "accept-1", "op": "accept", "B": 1, "gamma": 16, "V": 151936, "mix": "usual",
         "ragged": False, "len_seed": 0},
        # 32 requests with truncated blocks, settings of their own
        {"name": "accept-32-ragged", "op": "accept", "B": 32, "gamma": 16, "V": 151936,
         "mix": "mixed", "ragged": True, "len_seed": 1},
        # high concurrency, truncated blocks, top-p alone
        {"name": "accept-128-ragged", "op": "accept", "B": 128, "gamma": 16, "V": 129280,
         "mix": "top_p", "ragged": True, "len_seed": 2},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "product", "sample", "accept"])
    if op == "quantise":
        d = 32 * _log_int(rng, 2, 224)
        return {"op": op, "rows": _log_int(rng, 1, 100000), "d": d,
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "product":
        return {"op": op, "rows": _log_int(rng, 1, 1500), "d": 32 * _log_int(rng, 4, 224),
                "V": _log_int(rng, 1000, 129000), "out": rng.choice(["bf16", "fp32"])}
    mix = rng.choice(["usual", "mixed", "top_p", "min_p", "top_k", "plain"])
    if op == "sample":
        return {"op": op, "rows": _log_int(rng, 1, 800), "V": _log_int(rng, 1000, 151000),
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "mix": mix,
                "masked": rng.random() < 0.3}
    return {"op": op, "B": _log_int(rng, 1, 96), "gamma": rng.randint(1, 16),
            "V": _log_int(rng, 1000, 129000), "mix": mix, "ragged": rng.random() < 0.7,
            "len_seed": rng.randrange(1 << 20)}


def _lengths(case):
    """Kept drafts of each request: the gamma of a whole block, or a truncated prefix."""
    rng = random.Random(case["len_seed"])
    g = case["gamma"]
    if not case["ragged"]:
        return [g] * case["B"]
    return [min(g, int(rng.expovariate(1.0 / (0.4 * g + 0.5)))) for _ in range(case["B"])]


def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if op == "quantise":
        n = case["rows"] * case["d"]
        packed = n / 2 + n / BLOCK
        return {"bytes": n * size[case["dtype"]] + 2 * packed + 2 * n, "flops": 4 * n}
    if op == "product":
        m, d, v = case["rows"], case["d"], case["V"]
        return {"bytes": 2 * m * d + v * (d / 2 + d / BLOCK) + m * v * size[case["out"]],
                "flops": 2 * m * d * v}
    if op == "sample":
        n = case["rows"] * case["V"]
        return {"bytes": n * size[case["dtype"]] + 16 * case["rows"], "flops": 4 * n}
    kept = sum(_lengths(case))
    n = (kept + case["B"]) * case["V"]
    return {"bytes": 4 * n + 2 * kept * case["V"], "flops": 4 * n + 4 * kept * case["V"]}


# ------------------------------------------------------------------ inputs

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _settings(mix, n, gen):
    """Per-request temperature, top_k (0: off), top_p (1: off), min_p (0: off), on the GPU."""
    r = torch.rand((4, n), generator=gen)
    one = torch.ones(n)
    t, k, p, m = one.clone(), torch.zeros(n, dtype=torch.int32), one.clone(), 0 * one
    if mix == "usual":
        t, k, p = 0.8 * one, torch.full((n,), 50, dtype=torch.int32), 0.95 * one
    elif mix == "top_p":
        p = 0.85 + 0.1 * r[2]
    elif mix == "top_k":
        t, k = 0.7 * one, (1 + 400 * r[1] * r[1]).to(torch.int32)
    elif mix == "min_p":
        m = 0.02 + 0.1 * r[3]
    elif mix == "mixed":
        t = torch.where(r[0] < 0.1, 0 * one, 0.5 + 0.8 * r[0])
        k = torch.where(r[1] < 0.4, 0 * one, 1 + 1000 * (r[1] - 0.4) ** 2).to(torch.int32)
        p = torch.where(r[2] < 0.3, one, 0.7 + 0.3 * r[2])
        m = torch.where(r[3] < 0.6, 0 * one, 0.2 * (r[3] - 0.6))
    return [x.cuda() for x in (t.float(), k, p.float(), m.float())]


def _head(rows, V, gen):
    """Logits as a model's head makes them: a broad body and a few dozen likely ids."""
    z = torch.randn((rows, V), generator=gen, device="cuda") * 1.5
    ids = torch.randint(0, V, (rows, 48), generator=gen, device="cuda")
    z.scatter_add_(1, ids, 3 + 7 * torch.rand((rows, 48), generator=gen, device="cuda") ** 2)
    return z


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "quantise":
        s["x"] = torch.randn((case["rows"], case["d"]), generator=gen, device="cuda",
                             dtype=_TYPES[case["dtype"]])
    elif op == "product":
        s["hidden"] = torch.randn((case["rows"], case["d"]), generator=gen, device="cuda",
                                  dtype=torch.bfloat16)
        head = torch.randn((case["V"], case["d"]), generator=gen, device="cuda",
                           dtype=torch.bfloat16)
        code, exponent = _mx_parts(head)
        s["codes"], s["scales"] = _mx_pack(code, exponent)
    elif op == "sample":
        n, V = case["rows"], case["V"]
        z = _head(n, V, gen)
        if case["masked"]:
            # a grammar allows a few ids on every fourth row, none on the very last masked one
            banned = torch.rand((n, V), generator=gen, device="cuda") < 0.98
            rows = torch.arange(n, device="cuda") % 4 == 1
            z.masked_fill_(banned & rows[:, None], float("-inf"))
            z[(n - 2) // 4 * 4 + 1 if n >= 2 else 0] = float("-inf")
        s["logits"] = z.to(_TYPES[case["dtype"]])
        s["u"] = torch.rand(n, generator=gen, device="cuda")
        s["settings"] = _settings(case["mix"], n, host)
    else:
        B, g, V = case["B"], case["gamma"], case["V"]
        L = _lengths(case)
        starts = [0]
        for x in L:
            starts.append(starts[-1] + x + 1)
        s["lens"] = torch.tensor(L, dtype=torch.int32, device="cuda")
        s["offsets"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        base = _head(B * g, V, gen)
        noise = torch.randn((B * g, V), generator=gen, device="cuda")
        s["draft_logits"] = (base + 0.3 * noise).to(torch.bfloat16).view(B, g, V)
        s["settings"] = _settings(case["mix"], B, host)
        # drafted ids: among the drafter's likely ones, by a noisy argmax
        noise.exponential_(generator=gen).log_().neg_()
        s["tokens"] = (s["draft_logits"].float().view(B * g, V) + 0.5 * noise).argmax(1).to(
            torch.int32).view(B, g)
        noise.normal_(generator=gen)
        packed = torch.zeros((B * (g + 1), V), device="cuda")
        at = torch.cat([torch.arange(x, device="cuda") + st for x, st in zip(L, starts)])
        of = torch.cat([torch.arange(x, device="cuda") + r * g for r, x in enumerate(L)])
        packed[at] = base[of] + 0.3 * noise[of]
        packed[s["offsets"][1:].long() - 1] = _head(B, V, gen)      # the bonus rows
        s["logits"] = packed
        s["u_accept"] = torch.rand((B, g), generator=gen, device="cuda")
        s["u_resample"] = torch.rand((B, g + 1), generator=gen, device="cuda")
    if own:
        _own_prepare(s)
    return s


def run(s):
    if own:
        return _own_run(s)
    return {"quantise": _plain_quantise, "product": _plain_product, "sample": _plain_sample,
            "accept": _plain_accept}[s["case"]["op"]](s)


# ------------------------------------------------------------------ plain forms

def _mx_parts(x):
    """e2m1 codes (uint8, sign in bit 3) [rows][d] and scale exponents (int32) [rows][d/32]."""
    rows, d = x.shape
    b = x.float().view(rows, d // BLOCK, BLOCK)
    top = b.abs().amax(2)
    exponent = (torch.frexp(top)[1] - 3).clamp(-127, 127)      # floor(log2(top)) - 2
    exponent = torch.where(top > 0, exponent, torch.full_like(exponent, -127))
    y = torch.ldexp(b, -exponent[:, :, None].expand_as(b))
    a = y.abs()
    # round to nearest, ties to the even code: borders between neighbours of GRID
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8)
            + (a > 1.25).to(torch.uint8) + (a >= 1.75).to(torch.uint8)
            + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
            + (a > 5.0).to(torch.uint8))
    code = code + 8 * torch.signbit(y).to(torch.uint8)
    return code.view(rows, d), exponent.to(torch.int32)


def _mx_pack(code, exponent):
    """Two codes a byte, the even column in the low half; a scale is its exponent + 127."""
    return code[:, 0::2] | (code[:, 1::2] << 4), (exponent + 127).to(torch.uint8)


def _mx_values(code, exponent):
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=code.device)
    rows, d = code.shape
    v = grid[code.int()].view(rows, d // BLOCK, BLOCK)
    return torch.ldexp(v, exponent[:, :, None].expand_as(v)).view(rows, d)


def _mx_unpack(codes, scales):
    code = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1)
    return _mx_values(code, scales.to(torch.int32) - 127)


def _plain_quantise(s):
    return _mx_values(*_mx_parts(s["x"])).to(torch.bfloat16)     # every value is a bf16 number


def _plain_product(s):
    h = _mx_values(*_mx_parts(s["hidden"]))
    w = _mx_unpack(s["codes"], s["scales"])
    return (h @ w.t()).to(_TYPES[s["case"]["out"]])


def _filter(z, t, k, p, m):
    """(weights in id order with the filtered ids at 0, size of the kept set) of each row of z:
    softmax weights at temperature t over the k likeliest ids, of these the shortest leading
    run that holds a share p, of these the ones with at least m times the largest weight; the
    likeliest id stays. Equal logits rank by id; temperature 0 keeps the likeliest id alone."""
    z = torch.where(torch.isnan(z), float("-inf"), z.float())
    some = z.amax(1) > float("-inf")
    zs, order = torch.sort(z, dim=1, descending=True, stable=True)
    greedy = t <= 0
    td = torch.where(greedy, 1.0, t.double())
    w = torch.exp((zs.double() - zs[:, :1].double()) / td[:, None])
    w = torch.where(some[:, None], w, 0.0)
    rank = torch.arange(z.shape[1], device=z.device)[None, :]
    limit = torch.where(greedy, 1, torch.where(k > 0, k, z.shape[1]))
    keep = (rank < limit[:, None]) & (zs > float("-inf"))
    wk = torch.where(keep, w, 0.0)
    cum = torch.cumsum(wk, 1)
    share = (p.double()[:, None] * cum[:, -1:])
    keep &= (cum - wk < share) | (p >= 1)[:, None] | (rank == 0)
    keep &= (w >= m.double()[:, None]) | (rank == 0)
    keep &= some[:, None]
    out = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    return out, keep.sum(1)


def _inverse_cdf(w, u):
    """Smallest id whose running weight passes u times the total; -1 without any weight."""
    c = torch.cumsum(w, 1)
    hit = (c > u.double()[:, None] * c[:, -1:]) & (w > 0)
    ids = torch.arange(w.shape[1], device=w.device)
    last = torch.where(w > 0, ids, -1).amax(1)
    first = torch.where(hit, ids, w.shape[1]).amin(1)
    return torch.where(hit.any(1), first, last)


def _plain_sample(s):
    w, kept = _filter(s["logits"], *s["settings"])
    token = _inverse_cdf(w, s["u"])
    drawn = w.gather(1, token.clamp(min=0)[:, None])[:, 0]
    logprob = torch.where(token >= 0, torch.log(drawn / w.sum(1)), float("-inf"))
    return {"tokens": token.to(torch.int32), "kept": kept.to(torch.int32),
            "logprob": logprob.float()}


def _plain_accept(s):
    q, x, lens = s["draft_logits"], s["tokens"].long(), s["lens"].long()
    B, g, V = q.shape
    per_row = [a.repeat_interleave(g + 1) for a in s["settings"]]
    per_draft = [a.repeat_interleave(g) for a in s["settings"]]
    at = s["offsets"][:-1].long()[:, None] + torch.arange(g + 1, device="cuda")
    at = torch.minimum(at, s["offsets"][1:, None].long() - 1)
    wp = _filter(s["logits"][at.reshape(-1)], *per_row)[0]
    wp = (wp / wp.sum(1, keepdim=True)).view(B, g + 1, V)
    wq = _filter(q.reshape(B * g, V), *per_draft)[0]
    wq = (wq / wq.sum(1, keepdim=True)).view(B, g, V)
    px = wp[:, :g].gather(2, x[:, :, None])[:, :, 0]
    qx = wq.gather(2, x[:, :, None])[:, :, 0]
    live = torch.arange(g, device="cuda")[None, :] < lens[:, None]
    fails = ~(s["u_accept"].double() < torch.clamp(px / qx, max=1.0)) & live
    a = torch.where(fails.any(1), fails.int().argmax(1), lens)
    rows = torch.arange(B, device="cuda")
    p_a, q_a = wp[rows, a], wq[rows, a.clamp(max=g - 1)]
    w = torch.where((a < lens)[:, None], torch.clamp(p_a - q_a, min=0.0), p_a)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, p_a)
    token = _inverse_cdf(w, s["u_resample"][rows, a])
    return {"accept_len": a.to(torch.int32), "next_token": token.to(torch.int32)}


# ------------------------------------------------------------------ the library's calls

def _own_prepare(s):
    """What a program keeps between calls: weight handle, parameter handle, workspaces."""
    import draft_block_verification_amd as sd
    c, op = s["case"], s["case"]["op"]
    if op == "product":
        s["head"] = sd.Mxfp4Weights(s["codes"], s["scales"], c["d"])
        s["ws"] = sd.new_workspace(sd.mxfp4_logits_workspace_bytes(c["rows"], c["d"]), "cuda")
    elif op == "sample":
        s["params"] = sd.SamplingParams(*s["settings"])
        s["ws"] = sd.new_workspace(sd.sample_workspace_bytes(c["rows"], c["V"]), "cuda")
    elif op == "accept":
        s["params"] = sd.SamplingParams(*s["settings"])
        s["ws"] = sd.new_workspace(sd.accept_filtered_workspace_bytes(c["B"], c["gamma"], c["V"]),
                                   "cuda")


def _own_run(s):
    import draft_block_verification_amd as sd
    c, op = s["case"], s["case"]["op"]
    if op == "quantise":
        codes, scales = sd.sd_mxfp4_quantize(s["x"])
        return sd.sd_mxfp4_dequantize(codes, scales, c["d"], torch.bfloat16)
    if op == "product":
        return sd.sd_mxfp4_logits(s["hidden"], s["head"], dtype=_TYPES[c["out"]],
                                  workspace=s["ws"])
    if op == "sample":
        token, kept, logprob = sd.sd_sample(s["logits"], s["u"], s["params"], workspace=s["ws"])
        return {"tokens": token, "kept": kept, "logprob": logprob}
    a, token = sd.sd_accept_filtered(s["logits"], s["draft_logits"], s["tokens"], s["lens"],
                                     s["offsets"], s["u_accept"], s["u_resample"], s["params"],
                                     workspace=s["ws"])
    return {"accept_len": a, "next_token": token}


# ------------------------------------------------------------------ 64-bit statement

def _exact_mx(x):
    """Values of the MXFP4 form of x, in 64 bits: nearest grid point under the block's scale,
    by the distance to every grid point (ties go to the even code)."""
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 24) // x.shape[1])
    for r in range(0, x.shape[0], step):
        b = x[r:r + step].double().unflatten(1, (-1, BLOCK))
        top = b.abs().amax(2, keepdim=True)
        scale = 2.0 ** (torch.floor(torch.log2(top.clamp(min=2.0 ** -126))) - 2).clamp(-127, 127)
        a = (b.abs() / scale).clamp(max=6.0)
        lo = torch.bucketize(a, grid, right=True) - 1
        hi = (lo + 1).clamp(max=7)
        up, down = grid[hi] - a, a - grid[lo]
        code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        out[r:r + step] = (grid[code] * scale * torch.sign(b)).flatten(1)
    return out


def _exact_sample_row(z, u, t, k, p, m):
    """log-probability of the drawn id of one row, from the definition, on the host."""
    z = np.where(np.isnan(z), -np.inf, z)
    if z.max() == -np.inf:
        return -math.inf
    if t <= 0:
        return 0.0
    ids = np.flatnonzero(z > -np.inf)
    ids = ids[np.lexsort((ids, -z[ids]))]
    if k > 0:
        ids = ids[:k]
    w = np.exp((z[ids] - z[ids[0]]) / t)
    n = len(ids)
    if p < 1:
        n = min(n, max(1, int(np.searchsorted(np.cumsum(w), p * w.sum(), side="left")) + 1))
    if m > 0:
        n = min(n, max(1, int(np.count_nonzero(w >= m))))
    by_id = np.argsort(ids[:n])
    w = w[:n][by_id]
    c = np.cumsum(w)
    at = min(int(np.searchsorted(c, u * c[-1], side="right")), n - 1)
    return float(np.log(w[at] / w.sum()))


def exact(case, seed):
    op = case["op"]
    if op == "accept":
        return None             # whole numbers only
    if op == "sample" and case["rows"] * case["V"] > 2e7:
        return None             # minutes on the host
    s = prepare(case, seed)
    if op == "quantise":
        return _exact_mx(s["x"])
    if op == "product":
        h = _exact_mx(s["hidden"])
        c = s["codes"].long()
        grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
        out = torch.empty((case["rows"], case["V"]), dtype=torch.float64, device="cuda")
        for v in range(0, case["V"], 8192):
            part = torch.stack([c[v:v + 8192] % 16, c[v:v + 8192] // 16], 2).flatten(1)
            w = grid[part % 8] * (1.0 - 2.0 * (part // 8))
            e = s["scales"][v:v + 8192].double() - 127.0
            out[:, v:v + 8192] = h @ (w * (2.0 ** e).repeat_interleave(BLOCK, 1)).t()
        return out
    z = s["logits"].double().cpu().numpy()
    u = s["u"].double().cpu().numpy()
    t, k, p, m = (x.double().cpu().numpy() for x in s["settings"])
    lp = [_exact_sample_row(z[r], u[r], t[r], int(k[r]), p[r], m[r]) for r in range(len(z))]
    return {"tokens": None, "kept": None,
            "logprob": torch.tensor(lp, dtype=torch.float64)}
