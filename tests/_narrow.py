"""64-bit statements of the norm, of MXFP8 rows and of 4-bit integers with group scales (numpy,
written from the definitions), shared by the tests on the CPU and on the GPU."""
import numpy as np
import torch

E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)])[:127]


def rand(rows, d, dtype, seed, spread=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, d), generator=g)
    if spread:      # groups of very different size
        n = -(-d // 8)
        size = torch.exp2(torch.randint(-12, 12, (rows, n), generator=g).float())
        x = x * size.repeat_interleave(8, 1)[:, :d]
        if dtype == torch.float16:
            x = x.clamp(-60000, 60000)
    return x.to(dtype)


def padded(d):
    return -(-d // 128) * 128


def mx8_quantize(x):
    """codes [rows][kp], scale bytes [rows][kp / 32] of float64 rows."""
    rows, d = x.shape
    b = np.zeros((rows, padded(d)))
    b[:, :d] = x
    b = b.reshape(rows, -1, 32)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    top = np.abs(b).max(axis=2)
    e = np.where(top > 0, np.frexp(top)[1] - 1 - 8, -127)
    e = np.maximum(e, -127)
    y = b / 2.0 ** e[:, :, None]
    a = np.minimum(np.abs(y), 448.0)
    lo = np.searchsorted(E4M3, a, side="right") - 1
    hi = np.minimum(lo + 1, 126)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = code + np.where(np.signbit(y), 128, 0)
    code = np.where(bad[:, :, None], 0, code)
    return (code.reshape(rows, -1).astype(np.uint8),
            np.where(bad, 255, e + 127).astype(np.uint8))


def mx8_values(codes, scales, d):
    c = codes.astype(np.int64)
    v = np.append(E4M3, np.nan)[c % 128] * np.where(c >= 128, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v * np.repeat(s, 32, axis=1))[:, :d]


def to16(x, dtype):
    """float64 to fp32, then to a 16-bit torch type, as float64."""
    return torch.from_numpy(x.astype(np.float32)).to(dtype).double().numpy()


def w4_quantize(x, group, symmetric, dtype):
    """codes [rows][d / 2], scales (torch, dtype), zeros [rows][d / group] or None."""
    rows, d = x.shape
    b = x.reshape(rows, -1, group)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    up, down = np.maximum(b.max(axis=2), 0), np.maximum((-b).max(axis=2), 0)
    if symmetric:
        s = to16(np.float32(np.maximum(up, down)) / np.float32(7), dtype)
    else:
        s = to16((up + down) / 15, dtype)
    bad |= ~np.isfinite(s)
    none = ~bad & (s < 2.0 ** -126)
    one = np.where(bad | none, 1.0, s)
    quotient = lambda v: np.rint((v / one[..., None]).astype(np.float32).astype(np.float64))
    z = np.full(s.shape, 8.0) if symmetric else np.minimum(quotient(down[..., None])[..., 0], 15)
    if not symmetric:
        z = np.where(bad | none, 0.0, z)
    c = np.clip(quotient(b) + z[:, :, None], 0, 15)
    c = np.where((bad | none)[:, :, None], z[:, :, None], c).reshape(rows, d).astype(np.uint8)
    s = np.where(bad, np.nan, np.where(none, 0.0, s))
    return (c[:, 0::2] | c[:, 1::2] << 4, torch.from_numpy(s).to(dtype),
            None if symmetric else z.astype(np.uint8))


def w4_parts(codes, scales, zeros):
    """(codes - zeros), scales broadcast over the columns, and (codes + zeros), float64 [rows][d]."""
    c = np.stack([codes & 15, codes >> 4], axis=2).reshape(codes.shape[0], -1).astype(np.float64)
    s = scales.double().numpy()
    group = c.shape[1] // s.shape[1]
    z = np.full(s.shape, 8.0) if zeros is None else zeros.astype(np.float64)
    wide = lambda v: np.repeat(v, group, axis=1)
    return c - wide(z), wide(s), c + wide(z)


def norm(x, weight=None, residual=None, eps=1e-6, offset=0.0):
    """(sum in the residual's type, y in float64) of torch rows on the CPU."""
    s = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
    v = s.double().numpy()
    with np.errstate(all="ignore"):
        y = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + float(np.float32(eps)))
        if weight is not None:
            y = y * (weight.double().numpy() + float(np.float32(offset)))
    return s, y


def check_rounded(got, want, dtype, slack=0.0):
    """Every value of `got` within half a step of its type from `want` (float64), which may itself
    be `slack` off: an fp32 rounding may come before (2^-24), subnormals step in absolute size."""
    info = torch.finfo(dtype)
    w = torch.from_numpy(np.asarray(want))
    tiny = info.tiny * info.eps / 2
    half = info.eps / 2 if dtype != torch.float32 else 0.0
    tol = w.abs() * (half + 2.0 ** -24) * (1 + 1e-6) + slack + tiny
    g = got.double().cpu()
    same = (g == w) | (torch.isnan(g) & torch.isnan(w))
    over = torch.isinf(g) & (w.abs() >= info.max)
    assert bool((same | over | ((g - w).abs() <= tol)).all()), float(((g - w).abs() / tol).nan_to_num(0).max())
