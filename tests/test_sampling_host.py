"""Refusals and host-side logic of the MXFP4, sampling and filtered-acceptance calls: every
call below fails a check before the library touches the HIP runtime. The statements the GPU
tests compare with are checked against hand-worked values and brute force."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import _filtered as F
import draft_block_verification_amd as sd

lib = ctypes.CDLL(sd.LIB_PATH)
FAKE = ctypes.c_void_p(0x10000)          # aligned, never dereferenced on the host
ODD = ctypes.c_void_p(0x10001)
TWO = ctypes.c_void_p(0x10002)
i64, sz = ctypes.c_int64, ctypes.c_size_t


class Four(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in "abcd"]


def call(f, args, **change):
    args = dict(args)
    args.update(change)
    return f(*args.values())


def test_mxfp4_sizes():
    assert [sd.mxfp4_columns(d) for d in (8, 128, 136, 7168)] == [128, 128, 256, 7168]
    for d in (0, -8, 12, 1 << 21):
        with pytest.raises(ValueError):
            sd.mxfp4_columns(d)
        assert sd.mxfp4_logits_workspace_bytes(4, d) == 0
    assert sd.mxfp4_logits_workspace_bytes(0, 128) == 0
    assert sd.mxfp4_logits_workspace_bytes(5, 256) >= 256 + 5 * 128 + 5 * 8


@pytest.mark.parametrize("name", ["sd_mxfp4_quantize", "sd_mxfp4_dequantize"])
def test_mxfp4_rows_refusals(name):
    f = getattr(lib, name)
    if name.endswith("de" + "quantize"):
        ok = dict(codes=FAKE, scales=FAKE, rows=4, d=256, x=FAKE, type=0, stride=i64(256), stream=None)
    else:
        ok = dict(x=FAKE, type=0, rows=4, d=256, stride=i64(256), codes=FAKE, scales=FAKE, stream=None)
    for p in ("x", "codes", "scales"):
        assert call(f, ok, **{p: None}) == 1
    assert call(f, ok, type=3) == 1 and call(f, ok, type=-1) == 1
    assert call(f, ok, rows=0) == 2
    assert call(f, ok, d=0) == 2 and call(f, ok, d=12) == 2
    assert call(f, ok, stride=i64(255)) == 2 and call(f, ok, stride=i64(1 << 41)) == 2
    assert call(f, ok, rows=2 ** 31 - 1, d=1024, stride=i64(1024)) == 2
    assert call(f, ok, x=TWO) == 3 and call(f, ok, x=ODD, type=1) == 3
    assert call(f, ok, codes=ctypes.c_void_p(0x10008)) == 3 and call(f, ok, scales=TWO) == 3


def test_mxfp4_head_refusals():
    size = lib.sd_mxfp4_head_bytes
    size.restype = ctypes.c_size_t
    assert size(64, 128) == 4096 + 256 and size(65, 136) == 4 * (4096 + 256)
    assert size(0, 128) == size(5, 12) == size(5, 0) == size((1 << 21) + 1, 128) == 0
    f = lib.sd_mxfp4_head
    ok = dict(codes=FAKE, scales=FAKE, V=100, d=256, head=FAKE, n=sz(4 * 4352), stream=None)
    for p in ("codes", "scales", "head"):
        assert call(f, ok, **{p: None}) == 1
    assert call(f, ok, V=0) == 2 and call(f, ok, d=100) == 2
    assert call(f, ok, codes=ctypes.c_void_p(0x10008)) == 3 and call(f, ok, scales=TWO) == 3
    assert call(f, ok, head=ctypes.c_void_p(0x10010)) == 3
    assert call(f, ok, n=sz(4 * 4352 - 1)) == 4


def test_mxfp4_logits_refusals():
    f = lib.sd_mxfp4_logits
    ok = dict(hidden=FAKE, ht=1, M=3, d=256, hs=i64(256), head=FAKE, V=100, out=FAKE, ot=0,
              ld=i64(100), ws=FAKE, wsb=sz(1 << 20), stream=None)
    for p in ("hidden", "head", "out"):
        assert call(f, ok, **{p: None}) == 1
    assert call(f, ok, ht=5) == 1 and call(f, ok, ot=5) == 1
    assert call(f, ok, M=0) == 2 and call(f, ok, d=100) == 2 and call(f, ok, V=0) == 2
    assert call(f, ok, V=(1 << 21) + 1, ld=i64(1 << 22)) == 2
    assert call(f, ok, M=1 << 23, V=1 << 21, ld=i64(1 << 21), wsb=sz(1 << 40)) == 2
    assert call(f, ok, hs=i64(200)) == 2 and call(f, ok, ld=i64(99)) == 2
    assert call(f, ok, out=TWO) == 3 and call(f, ok, hidden=ODD) == 3
    assert call(f, ok, head=ctypes.c_void_p(0x10010)) == 3
    assert call(f, ok, ws=None) == 4 and call(f, ok, wsb=sz(300)) == 4
    assert call(f, ok, ws=ctypes.c_void_p(0x10040)) == 3


def test_sample_refusals():
    f = lib.sd_sample
    s = Four()
    ok = dict(z=FAKE, t=0, ld=i64(100), R=2, V=100, u=FAKE, s=ctypes.byref(s), per=1, x=FAKE, xs=i64(1),
              kept=None, lp=None, ws=FAKE, wsb=sz(1 << 26), stream=None)
    for p in ("z", "u", "s", "x"):
        assert call(f, ok, **{p: None}) == 1
    assert call(f, ok, t=4) == 1
    assert call(f, ok, R=0) == 2 and call(f, ok, V=0) == 2 and call(f, ok, V=1 << 22, ld=i64(1 << 22)) == 2
    assert call(f, ok, ld=i64(99)) == 2 and call(f, ok, per=0) == 2 and call(f, ok, xs=i64(0)) == 2
    assert call(f, ok, z=TWO) == 3 and call(f, ok, z=ODD, t=1) == 3 and call(f, ok, u=TWO) == 3
    assert call(f, ok, x=TWO) == 3 and call(f, ok, kept=TWO) == 3 and call(f, ok, lp=TWO) == 3
    assert call(f, ok, s=ctypes.byref(Four(0x10002))) == 3
    assert call(f, ok, ws=None) == 4 and call(f, ok, wsb=sz(10)) == 4
    assert call(f, ok, ws=ctypes.c_void_p(0x10040)) == 3
    assert sd.sample_workspace_bytes(0, 5) == sd.sample_workspace_bytes(5, 0) == 0
    assert sd.sample_workspace_bytes(5, (1 << 21) + 1) == 0 < sd.sample_workspace_bytes(5, 1 << 21)


def test_accept_filtered_refusals():
    f = lib.sd_accept_filtered
    s = Four()
    ok = dict(z=FAKE, q=FAKE, x=FAKE, vl=None, ro=None, ua=FAKE, ur=FAKE, s=ctypes.byref(s), B=2, g=4, V=100,
              a=FAKE, t=FAKE, c=None, ws=FAKE, wsb=sz(1 << 26), stream=None)
    for p in ("z", "q", "x", "ua", "ur", "s", "a", "t"):
        assert call(f, ok, **{p: None}) == 1
    assert call(f, ok, vl=FAKE) == 1 and call(f, ok, ro=FAKE) == 1
    assert call(f, ok, B=0) == 2 and call(f, ok, g=65) == 2 and call(f, ok, V=0) == 2
    for p in ("z", "q", "x", "ua", "ur", "a", "t", "c"):
        assert call(f, ok, **{p: TWO}) == 3
    assert call(f, ok, s=ctypes.byref(Four(None, 0x10002))) == 3
    assert call(f, ok, ws=None) == 4 and call(f, ok, wsb=sz(300)) == 4
    assert call(f, ok, ws=ctypes.c_void_p(0x10040)) == 3
    assert sd.accept_filtered_workspace_bytes(0, 4, 100) == 0


def test_binding_refusals_without_a_gpu():
    with pytest.raises(ValueError):
        sd.sd_mxfp4_quantize(torch.zeros(2, 32))              # a host tensor
    with pytest.raises(TypeError):
        sd.sd_mxfp4_quantize(torch.zeros(2, 32, dtype=torch.float64))
    with pytest.raises(TypeError):
        sd.sd_mxfp4_quantize(np.zeros((2, 32)))
    with pytest.raises(ValueError):
        sd.sd_sample(torch.zeros(2, 5), torch.zeros(2), sd.SamplingParams())
    for bad in (dict(temperature=-1.0), dict(temperature=float("inf")), dict(temperature=float("nan")),
                dict(top_p=float("nan")), dict(min_p=float("nan")), dict(top_k=1.5), dict(top_k=1 << 40),
                dict(top_k=[1, 2], top_p=[0.5]), dict(top_p=[]), dict(top_k=[3], n=2), dict(top_k=3, n=0)):
        with pytest.raises(ValueError):
            sd.SamplingParams(device="cpu", **bad)
    p = sd.SamplingParams(0.5, [1, 2, 3], None, 0.1, device="cpu")
    assert p.n == 3 and p.top_p is None and p.temperature.tolist() == [0.5] * 3
    assert sd.SamplingParams().n == 1


def test_flag_values():
    assert (sd.FLAG_SAMPLING, sd.FLAG_EMPTY_ROW) == (16, 32)


# ------------------------------------------------ the statements the GPU tests compare with

def test_statement_mxfp4_by_hand():
    x = np.zeros((1, 32))
    x[0, :8] = [6.0, 5.0, 3.5, 2.5, 1.75, 0.75, -0.25, -7.9]
    c, s = F.mx_quantize(x)
    assert s[0, 0] == 127 and s.shape == (1, 4) and c.shape == (1, 64)
    v = F.mx_values(c, s, 32)
    assert v[0, :8].tolist() == [6.0, 4.0, 4.0, 2.0, 2.0, 1.0, 0.0, -6.0]


def test_statement_filters_by_hand():
    z = np.log(np.array([0.1, 0.4, 0.05, 0.3, 0.15]))
    ids = lambda **k: np.flatnonzero(F.filtered(z, **k)[0]).tolist()
    assert ids() == [0, 1, 2, 3, 4]
    assert ids(k=2) == [1, 3]
    assert ids(p=0.5) == [1, 3] and ids(p=0.3) == [1] and ids(p=0.86) == [0, 1, 3, 4]
    assert ids(m=0.3) == [1, 3, 4]
    assert ids(k=3, p=0.8) == [1, 3]            # 0.4 + 0.3 of 0.85
    assert ids(t=0.0) == [1]
    assert F.filtered(np.zeros(7), k=3)[0].nonzero()[0].tolist() == [0, 1, 2]
    w, n = F.filtered(np.full(4, -np.inf))
    assert n == 0 and F.draw(w, 0.3) == -1


def test_statement_acceptance_is_lossless():
    """Over drafts drawn from q' and uniforms integrated out, the first emitted token follows
    p' exactly: sum over x of q'(x) [min(1, p'/q') at x, else the residual]."""
    r = np.random.default_rng(0)
    for k, p in itertools.product((0, 3), (1.0, 0.7)):
        z, zq = r.standard_normal(6) * 2, r.standard_normal(6) * 2
        wp, wq = F.filtered(z, 1.0, k, p)[0], F.filtered(zq, 1.0, k, p)[0]
        pp, qq = wp / wp.sum(), wq / wq.sum()
        keep = np.minimum(1.0, np.divide(pp, qq, out=np.zeros(6), where=qq > 0))
        res = np.maximum(pp - qq, 0)
        res = res / res.sum() if res.sum() > 0 else pp
        emitted = qq * keep + (qq * (1 - keep)).sum() * res
        assert np.allclose(emitted, pp, atol=1e-15)


def test_row_limits():
    """One call of the filtered samplers takes up to 2^22 rows."""
    assert sd.sample_workspace_bytes(1 << 22, 10) > 0 and sd.sample_workspace_bytes((1 << 22) + 1, 10) == 0
    assert sd.accept_filtered_workspace_bytes(1 << 15, 63, 10) > 0
    assert sd.accept_filtered_workspace_bytes(1 << 15, 64, 10) == 0
    assert sd.accept_filtered_workspace_bytes(1 << 24, 60, 10) == 0
    s = Four(None, None, None, None)
    args = [FAKE, 0, i64(10), (1 << 22) + 1, 10, FAKE, ctypes.byref(s), 1, FAKE, i64(1), None, None, FAKE,
            sz(1 << 40), None]
    assert lib.sd_sample(*args) == 2
    args = [FAKE] * 3 + [None, None, FAKE, FAKE, ctypes.byref(s), 1 << 15, 64, 10, FAKE, FAKE, None, FAKE,
                         sz(1 << 40), None]
    assert lib.sd_accept_filtered(*args) == 2
