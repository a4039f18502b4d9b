"""The ends of the MXFP4 and sampling calls' ranges on the GPU: rows of 2^21 ids, more than 2^31
elements a call, strides whose byte offsets pass 32 bits. Rows are compared with the 64-bit
statement one by one, those at the far end above all.

Tolerance: V weights are each rounded to units of 2^-b of the largest, b = 63 - log2 V (42 at 2^21),
so a sum is off by at most V 2^-(b+1) of the largest weight, that is (V 2^-(b+1)) / (sum / largest)
of itself. One id of two million may weigh no more than that, so a decision is compared with
the statement's at both ends of that interval: the size of the kept set with those of top-p a
tolerance less and more, the token with the ones drawn a tolerance earlier and later."""
import numpy as np
import pytest
import torch

import draft_block_verification_amd as sd
import _filtered as F

pytestmark = pytest.mark.gpu
V21 = 1 << 21


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    yield
    torch.cuda.empty_cache()


def sum_error(V, w):
    """Relative error of the library's sum of the weights w of a row of V ids."""
    return V * 2.0 ** (np.ceil(np.log2(V)) - 64) * w.max() / w.sum() + 1e-12


def leading(z, t, n):
    """Weights in id order of the first n ids of row z by rank."""
    w = np.zeros(len(z))
    ids = np.lexsort((np.arange(len(z)), -z))[:n]
    w[ids] = np.exp((z[ids] - z[ids[0]]) / t)
    return w


def kept_range(z, t, k, p, m):
    """Sizes of the kept set that top-p a sum's error less and more give."""
    if p == 1:
        return [F.filtered(z, t, k, p, m)[1]] * 2
    e = sum_error(len(z), F.filtered(z, t, k)[0])
    return [F.filtered(z, t, k, p + d, m)[1] for d in (-e, e)]


def drawn_between(w, u, error, token):
    """Whether token is one of those that uniforms within error of u draw."""
    return F.draw(w, max(u - error, 0.0)) <= int(token) <= F.draw(w, u + error)


def check_row(z, u, s, token, kept, logprob):
    """One row z (fp64) under s = (t, k, p, m): what the library gave, against the statement."""
    lo, hi = kept_range(z, *s)
    assert lo <= int(kept) <= hi
    w = leading(z, s[0], int(kept))
    e = sum_error(len(z), w)
    assert drawn_between(w, float(u), e, token)
    ref = np.log(w[int(token)] / w.sum())
    # one rounding to fp32, and a total within its error
    assert abs(float(logprob) - ref) <= 2.0 ** -24 * abs(ref) + 2 * e


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.75, 50, 0.953125, 0.0), (1.0, 0, 0.875, 0.0), (1.0, 0, 1.0, 0.0625),
            (1.0, 3000, 1.0, 0.0), (1.5, 200000, 0.75, 0.0)]


def as_params(settings):
    col = lambda i, dt: torch.tensor([s[i] for s in settings], dtype=dt, device="cuda")
    return sd.SamplingParams(col(0, torch.float32), col(1, torch.int32), col(2, torch.float32), col(3, torch.float32))


def likely(z, seed):
    """A few dozen likely ids in every row of z, in place."""
    g = torch.Generator("cuda").manual_seed(seed)
    ids = torch.randint(0, z.shape[1], (z.shape[0], 40), generator=g, device="cuda")
    z.scatter_(1, ids, (6 + 6 * torch.rand(ids.shape, generator=g, device="cuda")).to(z.dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [V21, V21 - 5, 300007])
def test_sample_longest_rows(V, dtype):
    """One row a request, dealt to several workgroups, rows half a billion elements apart."""
    R = len(SETTINGS)
    stride = (1 << 29) + 8 - V % 2             # the last row begins past 2^31 elements
    buf = torch.empty((R - 1) * stride + V, dtype=dtype, device="cuda")
    z = buf.as_strided((R, V), (stride, 1))
    g = torch.Generator("cuda").manual_seed(V)
    for r in range(R):
        z[r] = torch.randn(V, generator=g, device="cuda")
    likely(z, V + 1)
    u = torch.rand(R, generator=g, device="cuda")
    tokens = torch.full(((R - 1) * (1 << 28) + 1,), -7, dtype=torch.int32, device="cuda")
    out = tokens[::1 << 28]
    x, kept, lp = sd.sd_sample(z, u, as_params(SETTINGS), tokens=out)
    assert x.data_ptr() == tokens.data_ptr()
    for r in range(R):
        check_row(z[r].double().cpu().numpy(), u[r].cpu(), SETTINGS[r], x[r], kept[r], lp[r])
    assert bool((tokens[1:1 << 20] == -7).all()) and bool((tokens[-(1 << 20):-1] == -7).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_many_long_rows(dtype):
    """1100 rows of 2^21 ids: 2.3e9 logits, a workgroup a row."""
    R = 1100
    z = torch.empty((R, V21), dtype=dtype, device="cuda")
    g = torch.Generator("cuda").manual_seed(5)
    for r in range(0, R, 100):
        z[r:r + 100] = torch.randn((100, V21), generator=g, device="cuda")
    likely(z, 6)
    u = torch.rand(R, generator=g, device="cuda")
    settings = [SETTINGS[r % len(SETTINGS)] for r in range(R)]
    x, kept, lp = sd.sd_sample(z, u, as_params(settings))
    for r in [0, 1] + list(range(1022, 1028)) + list(range(R - 6, R)):
        check_row(z[r].double().cpu().numpy(), u[r].cpu(), settings[r], x[r], kept[r], lp[r])


@pytest.mark.parametrize("s", [SETTINGS[1], SETTINGS[2]])
def test_accept_longest_rows(s):
    """16 blocks of 64 drafts of 2^21 ids: 2.2e9 target and 2.1e9 drafter logits. The rows of both
    sides agree, so likely drafts are accepted up to the bonus row; one request draws a rejection
    at its last position instead, from a target that has the drafted id masked out."""
    B, g, V = 16, 64, V21
    gen = torch.Generator("cuda").manual_seed(9)
    z = torch.empty((B * (g + 1), V), device="cuda")
    q = torch.empty((B, g, V), dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        rows = z[b * (g + 1):(b + 1) * (g + 1)]
        rows[:] = torch.randn((g + 1, V), generator=gen, device="cuda").bfloat16().float()
        likely(rows, b)
        rows[:] = rows.bfloat16().float()
        q[b] = rows[:g].bfloat16()
    x = q.float().argmax(2).int()
    no = B - 2
    z[no * (g + 1) + g - 1, x[no, g - 1].long()] = -np.inf
    ua = 0.999 * torch.rand((B, g), generator=gen, device="cuda")
    ur = torch.rand((B, g + 1), generator=gen, device="cuda")
    a, t = sd.sd_accept_filtered(z, q, x, None, None, ua, ur, sd.SamplingParams(*s, n=B))
    assert a.tolist() == [g - (b == no) for b in range(B)]
    for b in (0, B // 2, no, B - 1):
        acc = int(a[b])
        zp = z[b * (g + 1) + acc].double().cpu().numpy()
        lo, hi = kept_range(zp, *s)
        u, got, fits = float(ur[b, acc]), int(t[b]), False
        for n in range(lo, hi + 1):
            w = leading(zp, s[0], n)
            e = sum_error(V, w)
            w /= w.sum()
            if acc == g:
                fits |= drawn_between(w, u, e, got)
                continue
            zq = q[b, acc].double().cpu().numpy()
            for nq in range(kept_range(zq, *s)[0], kept_range(zq, *s)[1] + 1):
                wq = leading(zq, s[0], nq)
                # a p' or q' off by e of itself moves a running sum of the residual by e at most
                r = np.maximum(w - wq / wq.sum(), 0.0)
                fits |= drawn_between(r, u, 2 * (e + sum_error(V, wq)) / r.sum(), got)
        assert hi - lo <= 3 and fits
    del z, q


def test_quantise_past_32_bits():
    """2.2e9 values in one call, and rows whose offsets pass 2^31 elements."""
    rows, d = 270001, 8192
    x = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator("cuda").manual_seed(3)
    for r in range(0, rows, 30000):
        x[r:r + 30000] = torch.randn(x[r:r + 30000].shape, generator=g, device="cuda")
    codes, scales = sd.sd_mxfp4_quantize(x)
    back = sd.sd_mxfp4_dequantize(codes, scales, d, torch.bfloat16)
    for r in (0, 131071, 131072, 262143, 262144, rows - 1):
        rc, rs = F.mx_quantize(x[r:r + 1].double().cpu().numpy())
        assert np.array_equal(codes[r].cpu().numpy(), rc[0]) and np.array_equal(scales[r].cpu().numpy(), rs[0])
        assert np.array_equal(back[r].double().cpu().numpy(), F.mx_values(rc, rs, d)[0])
    del x, back
    stride, R = (1 << 30) + 3, 4
    wide = torch.empty((R - 1) * stride + 136, dtype=torch.float16, device="cuda").as_strided((R, 136), (stride, 1))
    wide.copy_(torch.randn((R, 136), generator=g, device="cuda"))
    codes, scales = sd.sd_mxfp4_quantize(wide)
    rc, rs = F.mx_quantize(wide.double().cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    sd.sd_mxfp4_dequantize(codes, scales, 136, out=wide)
    assert np.array_equal(wide.double().cpu().numpy(), F.mx_values(rc, rs, 136).astype(np.float16).astype(float))


def logits_ref(h, codes, scales, ids, d):
    hv = F.mx_values(*F.mx_quantize(h.double().cpu().numpy()), d)
    wv = F.mx_values(codes[ids].cpu().numpy(), scales[ids].cpu().numpy(), d)
    return hv @ wv.T, np.abs(hv) @ np.abs(wv).T


def random_head(V, d, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    codes = torch.randint(0, 1 << 30, (V, d // 8), generator=g, device="cuda", dtype=torch.int32)
    codes ^= codes << 17
    return codes.view(torch.uint8), torch.randint(122, 130, (V, d // 32), generator=g, device="cuda", dtype=torch.uint8)


@pytest.mark.parametrize("M", [3, 40, 200])
def test_logits_of_a_head_past_32_bits(M):
    """An LM head of 2^21 ids whose codes take 2.7 GB, hidden rows and logits far apart."""
    V, d = V21, 2560
    codes, scales = random_head(V, d, M)
    h = torch.randn((M, d), generator=torch.Generator("cuda").manual_seed(M), device="cuda").bfloat16()
    head = sd.Mxfp4Weights(codes, scales, d)
    stride = (1 << 31) // max(M - 1, 2) + 8
    stride = max(stride, V + 8)
    buf = torch.full(((M - 1) * stride + V + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf.as_strided((M, V), (stride, 1))
    sd.sd_mxfp4_logits(h, head, out)
    ids = torch.cat([torch.arange(64), torch.arange(V - 300, V), torch.arange(1 << 20, (1 << 20) + 64)]).cuda()
    want, size = logits_ref(h, codes, scales, ids, d)
    got = out[:, ids].double().cpu().numpy()
    tol = d * 2.0 ** -24 * size
    tol = tol + (np.abs(want) + tol) * 2.0 ** -8
    assert (np.abs(got - want) <= tol).all()
    assert bool((buf[-8:] == 7).all()) and bool((out.as_strided((M - 1, 8), (stride, 1), V) == 7).all())


def test_logits_past_32_bits():
    """1100 rows by 2^21 ids: 2.3e9 logits."""
    M, V, d = 1100, V21, 128
    codes, scales = random_head(V, d, 1)
    h = torch.randn((M, d), generator=torch.Generator("cuda").manual_seed(2), device="cuda").bfloat16()
    out = sd.sd_mxfp4_logits(h, sd.Mxfp4Weights(codes, scales, d), dtype=torch.float16)
    ids = torch.cat([torch.arange(100), torch.arange(V - 300, V)]).cuda()
    rows = torch.tensor([0, 1, 500, 1023, 1024, 1025, M - 1]).cuda()
    want, size = logits_ref(h[rows], codes, scales, ids, d)
    got = out[rows][:, ids].double().cpu().numpy()
    tol = d * 2.0 ** -24 * size
    tol = tol + (np.abs(want) + tol) * 2.0 ** -11
    assert (np.abs(got - want) <= tol).all()
