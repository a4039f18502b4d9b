"""Refusals and host-side logic of the norm, MXFP8 and 4-bit integer calls: every call below fails
a check before the library touches the HIP runtime. The statements the GPU tests compare with are
checked against hand-worked values."""
import ctypes

import numpy as np
import pytest
import torch

import _narrow as N
import draft_block_verification_amd as sd

lib = ctypes.CDLL(sd.LIB_PATH)
FAKE = ctypes.c_void_p(0x10000)          # aligned, never dereferenced on the host
EIGHT, TWO, ODD = (ctypes.c_void_p(0x10000 + k) for k in (8, 2, 1))
OTHER = ctypes.c_void_p(0x20000)
i64, sz, f32 = ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
for _f in ("sd_mxfp8_head_bytes", "sd_mxfp8_logits_workspace_bytes", "sd_w4_head_bytes", "sd_w4_logits_workspace_bytes"):
    getattr(lib, _f).restype = sz
EINVAL, ESHAPE, EALIGN, EWORKSPACE = 1, 2, 3, 4


def call(f, args, **change):
    args = dict(args)
    args.update(change)
    return f(*args.values())


def norm_args(**tail):
    return dict(x=FAKE, xt=1, xs=i64(256), res=FAKE, rt=1, rs=i64(256), w=FAKE, wt=1, off=f32(0), eps=f32(1e-6), rows=4,
                d=256, sum=FAKE, ss=i64(256), **tail, stream=None)


@pytest.mark.parametrize("mx", [False, True])
def test_norm_refusals(mx):
    f = lib.sd_rms_norm_mxfp8 if mx else lib.sd_rms_norm
    ok = norm_args(codes=FAKE, scales=FAKE) if mx else norm_args(y=OTHER, yt=1, ys=i64(256))
    for p in ("x", "codes", "scales") if mx else ("x", "y"):
        assert call(f, ok, **{p: None}) == EINVAL
    for p in ("xt", "wt") + (() if mx else ("yt",)):
        for t in (-1, 3, 7):
            assert call(f, ok, **{p: t}) == EINVAL
    assert call(f, ok, rt=2) == EINVAL and call(f, ok, xt=0, rt=1) == EINVAL and call(f, ok, rt=3) == EINVAL
    assert call(f, ok, res=None) == EINVAL                               # a sum without a residual
    if not mx:
        assert call(f, ok, y=EIGHT, sum=EIGHT) == EINVAL                 # two results in one place
    for bad in (float("nan"), float("inf"), -1e-9):
        assert call(f, ok, eps=f32(bad)) == EINVAL
    for bad in (float("nan"), -float("inf")):
        assert call(f, ok, off=f32(bad)) == EINVAL
    assert call(f, ok, rows=0) == ESHAPE and call(f, ok, rows=-1) == ESHAPE
    assert call(f, ok, d=0) == ESHAPE and call(f, ok, d=(1 << 20) + 8, xs=i64(1 << 21), rs=i64(1 << 21)) == ESHAPE
    for p in ("xs", "rs", "ss") + (() if mx else ("ys",)):
        assert call(f, ok, **{p: i64(255)}) == ESHAPE and call(f, ok, **{p: i64((1 << 40) + 1)}) == ESHAPE
    for p in ("x", "res", "w", "sum") + (() if mx else ("y",)):
        assert call(f, ok, **{p: ODD}) == EALIGN
    if mx:
        assert call(f, ok, d=252) == ESHAPE
        assert call(f, ok, codes=EIGHT) == EALIGN and call(f, ok, scales=TWO) == EALIGN


@pytest.mark.parametrize("name", ["sd_mxfp8_quantize", "sd_mxfp8_dequantize"])
def test_mxfp8_rows_refusals(name):
    f = getattr(lib, name)
    if name.endswith("de" + "quantize"):
        ok = dict(codes=FAKE, scales=FAKE, rows=4, d=256, x=FAKE, type=0, stride=i64(256), stream=None)
    else:
        ok = dict(x=FAKE, type=0, rows=4, d=256, stride=i64(256), codes=FAKE, scales=FAKE, stream=None)
    for p in ("x", "codes", "scales"):
        assert call(f, ok, **{p: None}) == EINVAL
    assert call(f, ok, type=3) == EINVAL and call(f, ok, type=-1) == EINVAL
    assert call(f, ok, rows=0) == ESHAPE
    assert call(f, ok, d=0) == ESHAPE and call(f, ok, d=12) == ESHAPE
    assert call(f, ok, stride=i64(255)) == ESHAPE and call(f, ok, stride=i64(1 << 41)) == ESHAPE
    assert call(f, ok, rows=2 ** 31 - 1, d=1024, stride=i64(1024)) == ESHAPE
    assert call(f, ok, x=TWO) == EALIGN and call(f, ok, x=ODD, type=1) == EALIGN
    assert call(f, ok, codes=EIGHT) == EALIGN and call(f, ok, scales=TWO) == EALIGN


def test_mxfp8_head_and_logits_refusals():
    size = lib.sd_mxfp8_head_bytes
    assert size(64, 128) == 8192 + 256 and size(65, 136) == 4 * (8192 + 256)
    for V, d in ((0, 128), (1 << 22, 128), (64, 12), (64, 0), (64, (1 << 20) + 8), (1 << 21, 1 << 20)):
        assert size(V, d) == 0
    ok = dict(codes=FAKE, scales=FAKE, V=64, d=128, head=FAKE, bytes=sz(1 << 30), stream=None)
    for p in ("codes", "scales", "head"):
        assert call(lib.sd_mxfp8_head, ok, **{p: None}) == EINVAL
    assert call(lib.sd_mxfp8_head, ok, V=0) == ESHAPE and call(lib.sd_mxfp8_head, ok, d=12) == ESHAPE
    assert call(lib.sd_mxfp8_head, ok, bytes=sz(8192 + 255)) == EWORKSPACE
    for p, q in (("codes", EIGHT), ("scales", TWO), ("head", ctypes.c_void_p(0x10080))):
        assert call(lib.sd_mxfp8_head, ok, **{p: q}) == EALIGN

    need = lib.sd_mxfp8_logits_workspace_bytes
    assert need(5, 256) >= 256 + 5 * 256 + 5 * 8 and need(0, 128) == 0 and need(4, 12) == 0
    f = lib.sd_mxfp8_logits
    ok = dict(h=FAKE, ht=1, hs=None, M=5, d=256, stride=i64(256), head=FAKE, V=100, z=FAKE, zt=0, ld=i64(100), ws=FAKE,
              wb=sz(1 << 30), stream=None)
    coded = dict(ok, ht=3, hs=FAKE)
    for a in (ok, coded):
        for p in ("h", "head", "z"):
            assert call(f, a, **{p: None}) == EINVAL
        assert call(f, a, zt=3) == EINVAL
        assert call(f, a, M=0) == ESHAPE and call(f, a, V=0) == ESHAPE and call(f, a, d=100) == ESHAPE
        assert call(f, a, stride=i64(255)) == ESHAPE and call(f, a, ld=i64(99)) == ESHAPE
        assert call(f, a, z=TWO) == EALIGN and call(f, a, head=ctypes.c_void_p(0x10080)) == EALIGN
        assert call(f, a, wb=sz(need(5, 256) - 1)) == EWORKSPACE and call(f, a, ws=None) == EWORKSPACE
        assert call(f, a, ws=ctypes.c_void_p(0x10080)) == EALIGN
    assert call(f, ok, ht=4) == EINVAL and call(f, ok, ht=-1) == EINVAL
    assert call(f, ok, hs=FAKE) == EINVAL and call(f, coded, hs=None) == EINVAL
    assert call(f, ok, h=ODD) == EALIGN and call(f, coded, h=EIGHT) == EALIGN and call(f, coded, hs=TWO) == EALIGN
    assert call(f, coded, stride=i64(384)) == ESHAPE
    assert call(f, ok, M=1 << 22, V=1 << 17, ld=i64(1 << 17), wb=sz(1 << 50)) == ESHAPE


def test_w4_refusals():
    q = dict(x=FAKE, xt=1, rows=4, d=256, stride=i64(256), group=64, codes=FAKE, scales=FAKE, st=1, zeros=FAKE, stream=None)
    d = dict(codes=FAKE, scales=FAKE, st=1, zeros=FAKE, rows=4, d=256, group=64, x=FAKE, xt=1, stride=i64(256), stream=None)
    for f, ok in ((lib.sd_w4_quantize, q), (lib.sd_w4_dequantize, d)):
        for p in ("x", "codes", "scales"):
            assert call(f, ok, **{p: None}) == EINVAL
        assert call(f, ok, xt=3) == EINVAL and call(f, ok, st=0) == EINVAL and call(f, ok, st=3) == EINVAL
        for g in (0, 16, 48, 256, -32):
            assert call(f, ok, group=g) == ESHAPE
        assert call(f, ok, rows=0) == ESHAPE and call(f, ok, d=224) == ESHAPE and call(f, ok, d=0) == ESHAPE
        assert call(f, ok, stride=i64(255)) == ESHAPE
        assert call(f, ok, d=1 << 21, stride=i64(1 << 21)) == ESHAPE
        assert call(f, ok, rows=2 ** 31 - 1, d=1024, stride=i64(1024)) == ESHAPE
        for p, v in (("x", ODD), ("codes", EIGHT), ("scales", TWO), ("zeros", TWO)):
            assert call(f, ok, **{p: v}) == EALIGN
    size = lib.sd_w4_head_bytes
    assert size(64, 128, 128, 0) == 4096 + 128 and size(64, 128, 32, 1) == 4096 + 4 * 192 and size(65, 160, 32, 0) == 4 * (4096 + 512)
    for a in ((0, 128, 128, 0), (64, 96, 64, 0), (64, 128, 16, 0), (64, 128, 128, 2), (1 << 22, 128, 128, 0), (64, 1 << 21, 128, 0)):
        assert size(*a) == 0
    f = lib.sd_w4_head
    ok = dict(codes=FAKE, scales=FAKE, st=1, zeros=FAKE, V=64, d=128, group=128, head=FAKE, bytes=sz(1 << 30), stream=None)
    for p in ("codes", "scales", "head"):
        assert call(f, ok, **{p: None}) == EINVAL
    assert call(f, ok, st=0) == EINVAL and call(f, ok, group=96) == ESHAPE and call(f, ok, V=0) == ESHAPE
    assert call(f, ok, bytes=sz(4096 + 191)) == EWORKSPACE
    for p, v in (("codes", EIGHT), ("scales", TWO), ("zeros", TWO), ("head", ctypes.c_void_p(0x10080))):
        assert call(f, ok, **{p: v}) == EALIGN
    need = lib.sd_w4_logits_workspace_bytes
    assert need(5, 160, 32) >= 256 + 5 * 256 * 2 and need(0, 128, 128) == 0 and need(4, 96, 64) == 0
    f = lib.sd_w4_logits
    ok = dict(h=FAKE, ht=1, M=5, d=256, stride=i64(256), head=FAKE, V=100, group=64, st=1, hz=1, z=FAKE, zt=0, ld=i64(100),
              ws=FAKE, wb=sz(1 << 30), stream=None)
    for p in ("h", "head", "z"):
        assert call(f, ok, **{p: None}) == EINVAL
    for change in (dict(ht=0), dict(ht=3), dict(zt=3), dict(st=0), dict(hz=2), dict(hz=-1)):
        assert call(f, ok, **change) == EINVAL
    for change in (dict(M=0), dict(V=0), dict(group=96), dict(d=224), dict(stride=i64(255)), dict(ld=i64(99)),
                   dict(M=1 << 22, V=1 << 17, ld=i64(1 << 17), wb=sz(1 << 50))):
        assert call(f, ok, **change) == ESHAPE
    for change in (dict(h=ODD), dict(z=TWO), dict(head=ctypes.c_void_p(0x10080)), dict(ws=ctypes.c_void_p(0x10080))):
        assert call(f, ok, **change) == EALIGN
    assert call(f, ok, wb=sz(need(5, 256, 64) - 1)) == EWORKSPACE and call(f, ok, ws=None) == EWORKSPACE


def test_binding_refusals():
    """Tensors that are not on a device, of other types or shapes, settings out of range."""
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for f in (sd.sd_rms_norm, sd.sd_rms_norm_mxfp8, sd.sd_mxfp8_quantize, sd.sd_w4_quantize):
        with pytest.raises(ValueError):
            f(x)
        with pytest.raises(TypeError):
            f(x.to(torch.float64))
        with pytest.raises(TypeError):
            f([1.0])
    for f, a in ((sd.sd_mxfp8_dequantize, (x.byte(), x.byte(), 64)), (sd.sd_w4_dequantize, (x.byte(), x, None, 64))):
        with pytest.raises(ValueError):
            f(*a)
    for f in (sd.sd_mxfp8_logits, sd.sd_w4_logits):
        with pytest.raises((TypeError, ValueError)):
            f(x, x)
    with pytest.raises(ValueError):
        sd.RmsNorm(torch.ones(4))
    with pytest.raises(TypeError):
        sd.RmsNorm([1.0])
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(weight_offset=float("inf"))):
        with pytest.raises(ValueError):
            sd.RmsNorm(**bad)
    n = sd.RmsNorm(eps=1e-5, weight_offset=1.0)
    assert (n.eps, n.weight_offset, n.weight) == (1e-5, 1.0, None)
    with pytest.raises(AttributeError):
        n.eps = 2.0


def test_statement_of_mxfp8():
    x = np.zeros((1, 32))
    x[0, :8] = [256, 1, -1, 448, 470, 511, 17, 19]            # exponent 0: steps of 2 at 16 .. 32
    codes, scales = N.mx8_quantize(x)
    assert scales.tolist() == [[127, 0, 0, 0]]
    assert N.mx8_values(codes, scales, 8).tolist() == [[256, 1, -1, 448, 448, 448, 16, 20]]
    assert codes[0, :4].tolist() == [0x78, 0x38, 0xb8, 0x7e]
    tiny = N.mx8_quantize(np.full((1, 32), 2.0 ** -149))
    assert tiny[1][0, 0] == 0 and tiny[0][0, 0] == 0         # 2^-149 is an eighth of the least step
    bad = N.mx8_quantize(np.array([[np.nan] + [1.0] * 31]))
    assert bad[1][0, 0] == 255 and not bad[0].any()


def test_statement_of_w4():
    x = np.tile(np.arange(16.0) - 5, 2)[None]
    codes, scales, zeros = N.w4_quantize(x, 32, False, torch.bfloat16)
    assert scales.item() == 1 and zeros.item() == 5
    c, s, both = N.w4_parts(codes, scales, zeros)
    assert np.array_equal(c * s, x) and np.array_equal(both - c, np.full((1, 32), 10.0))
    assert codes[0, 0] == 0x10 and codes[0, 7] == 0xfe
    codes, scales, zeros = N.w4_quantize(x * 0.7, 32, True, torch.float16)
    assert zeros is None and scales.item() == np.float16(np.float32(7) / np.float32(7))
    z = N.w4_quantize(np.zeros((1, 32)), 32, False, torch.bfloat16)
    assert z[1].item() == 0 and z[2].item() == 0 and not z[0].any()
    bad = N.w4_quantize(np.array([[np.inf] + [1.0] * 31]), 32, True, torch.bfloat16)
    assert torch.isnan(bad[1]).all() and (bad[0] == 0x88).all()


def test_statement_of_the_norm():
    x = torch.tensor([[3.0, 4.0]])
    s, y = N.norm(x, torch.tensor([1.0, 0.0]), torch.tensor([[0.0, 0.0]]), 0.0, 1.0)
    assert torch.equal(s, x)
    assert np.allclose(y, [[2 * 3 / np.sqrt(12.5), 4 / np.sqrt(12.5)]], rtol=1e-15)
