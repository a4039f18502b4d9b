"""How far the seeded cases of test_gpu_sample.py lie from where the library may decide otherwise
than the 64-bit statement they are compared with: every decision of theirs, checked on the host.

The library's weights are good to 4e-14 and rounded to units of 2^-b of the row's largest, b = 46 or
63 - ceil(log2 V) if that is less. A sum over V ids is therefore off by at most V 2^-(b+1) of
the largest weight, which relative to the sum is `sum_error`. Decisions compared with it: top-p's
share against the running shares, the uniform against the kept set's running shares, the
acceptance probability against its uniform, the residual's running sum against its uniform
(residuals in units of 2^-51 besides). min-p's are single weights, good to 1e-13. The cases are run
up to the point where they would go to the GPU, and what they hold then is examined."""
import itertools

import numpy as np
import pytest
import torch

import _filtered as F
import test_gpu_sample as cases


class Held(Exception):
    """What a case was about to compare."""


class HostTorch:
    """torch, with tensors that ask for a device made on the host."""

    def __getattr__(self, name):
        return getattr(torch, name)

    @staticmethod
    def tensor(*args, device=None, **kwargs):
        return torch.tensor(*args, **kwargs)


def held(monkeypatch, name, kwargs):
    """(kind, arguments) that the GPU test `name` compares under parameters kwargs."""
    def stop(kind):
        def f(*args, **kw):
            raise Held(kind, args)
        return f
    monkeypatch.setattr(cases, "check_rows", stop("rows"))
    monkeypatch.setattr(F, "accept", stop("accept"))
    monkeypatch.setattr(cases, "torch", HostTorch())
    monkeypatch.setattr(cases.sd, "SamplingParams", lambda *a, **k: None)
    monkeypatch.setattr(torch.Tensor, "cuda", lambda t: t)
    with pytest.raises(Held) as e:
        getattr(cases, name)(**kwargs)
    return e.value.args


def parameters(name):
    """Every combination of the GPU test's parameters."""
    axes = []
    for m in getattr(getattr(cases, name), "pytestmark", []):
        if m.name == "parametrize":
            names = [n.strip() for n in m.args[0].split(",")]
            axes.append([dict(zip(names, v if len(names) > 1 else [v])) for v in m.args[1]])
    for choice in itertools.product(*axes):
        yield {k: v for part in choice for k, v in part.items()}


def sum_error(V, w):
    return V * 2.0 ** max(-47.0, np.ceil(np.log2(V)) - 64) * w.max() / w.sum() + 1e-13


def steps_from(w, u):
    """Distance of u from the running shares of w (id order) between its first and last id."""
    c = np.cumsum(w[w > 0])
    return np.min(np.abs(c[:-1] / c[-1] - u), initial=1.0)


def check_cut(z, s):
    """The row's cut lies off its borders."""
    t, k, p, m = s
    z = np.where(np.isnan(z), -np.inf, z)
    if z.max() == -np.inf or t == 0 or k == 1 or p <= 0:
        return
    zz = -np.sort(-z[z > -np.inf])[:k if k > 0 else None]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(zz == zz[0], 1.0, np.exp((zz - zz[0]) / t))
    if p < 1:
        assert np.min(np.abs(np.cumsum(w) / w.sum() - p)) > sum_error(len(z), w)
    if 0 < m < 1:
        assert np.min(np.abs(w / m - 1)) > 1e-13


ROWS = ["test_sample_settings", "test_sample_types_and_mixed_settings", "test_sample_many_rows",
        "test_sample_misleading_rows", "test_sample_three_filters"]
BLOCKS = ["test_accept_filtered", "test_accept_filtered_long_rows", "test_accept_filtered_three_filters",
          "test_accept_filtered_tokens_at_the_border", "test_accept_filtered_own_settings_and_hard_rows"]


@pytest.mark.parametrize("name", ROWS)
def test_sampled_rows(name, monkeypatch):
    for kwargs in parameters(name):
        kind, args = held(monkeypatch, name, kwargs)
        assert kind == "rows"
        z, u, settings = args[:3]
        z = torch.from_numpy(z).to(args[4] if len(args) > 4 else torch.float32).double().numpy()
        for r in range(len(z)):
            check_cut(z[r], settings[r])
            w, n = F.filtered(z[r], *settings[r])
            if n > 1:
                assert steps_from(w, float(u[r])) > sum_error(z.shape[1], w)


@pytest.mark.parametrize("name", BLOCKS)
def test_accepted_blocks(name, monkeypatch):
    for kwargs in parameters(name):
        with monkeypatch.context() as patch:
            kind, args = held(patch, name, kwargs)
        assert kind == "accept"
        z, zq, x, lens, offs, ua, ur, settings = args
        V = z.shape[1]
        for r in range(len(x)):
            s, a = settings[r], lens[r]
            for j in range(lens[r]):
                wp, wq = F.filtered(z[offs[r] + j], *s)[0], F.filtered(zq[r, j], *s)[0]
                check_cut(z[offs[r] + j], s)
                check_cut(zq[r, j], s)
                p = wp[x[r, j]] / wp.sum() if 0 <= x[r, j] < V and wp.sum() > 0 else 0.0
                q = wq[x[r, j]] / wq.sum() if 0 <= x[r, j] < V else 0.0
                # p and q off by e of themselves; where both are the same row's they are equal
                keep = 0.0 if p == 0 else 1.0 if p >= q else p / q
                if 0 < p < q:
                    assert abs(keep - ua[r, j]) > sum_error(V, wp) + sum_error(V, wq)
                if not ua[r, j] < keep:
                    a = j
                    break
            wp = F.filtered(z[offs[r] + a], *s)[0]
            if wp.sum() == 0:
                continue
            check_cut(z[offs[r] + a], s)
            w, e = wp / wp.sum(), sum_error(V, wp) + V * 2.0 ** -52
            if a < lens[r]:
                wq = F.filtered(zq[r, a], *s)[0]
                left = np.maximum(w - (wq / wq.sum() if wq.sum() > 0 else 0.0), 0.0)
                if left.sum() > 0:
                    w, e = left, (e + sum_error(V, wq)) / left.sum()
            if np.count_nonzero(w) > 1:
                assert steps_from(w, float(ur[r, a])) > e
