"""Filtered sampling and acceptance at the ends of their ranges, on the GPU against the 64-bit
statement: runs that end among ids of next to no weight, thresholds under the binned range.

Decisions are whole numbers and must be equal. Every drafted token and uniform here is chosen
so that the statement's decision holds by a wide margin (stated in each test), far over the
sums' error: a weight's rounding is half a unit of 2^-46 of the largest, V 2^-47 of the total
at the most (2e-10 for the 30011 ids of the longest row), and 4e-14 of each weight."""
import numpy as np
import pytest
import torch

import draft_block_verification_amd as sd
import _filtered as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    yield


def accept(z, zq, x, ua, ur, settings):
    """(accept_len, next_token) of the library and of the statement, whole blocks."""
    B, g, V = zq.shape
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    zqb = torch.from_numpy(zq).to(torch.bfloat16)
    col = lambda i, dt: torch.tensor([s[i] for s in settings], dtype=dt, device="cuda")
    params = sd.SamplingParams(col(0, torch.float32), col(1, torch.int32), col(2, torch.float32),
                               col(3, torch.float32))
    got = sd.sd_accept_filtered(c(z.reshape(-1, V)), zqb.cuda(), c(x), None, None, c(ua), c(ur), params)
    offs = np.arange(B + 1) * (g + 1)
    want = F.accept(z.reshape(-1, V).astype(np.float64), zqb.double().numpy(), x, [g] * B, offs, ua, ur, settings)
    return [t.cpu().tolist() for t in got], [w.tolist() for w in want]


@pytest.mark.parametrize("T", [1.0, 0.25, 3.0])
@pytest.mark.parametrize("bulk", ["one value", "few values", "spread"])
@pytest.mark.parametrize("V", [5000, 30011])       # a workgroup a row; several
def test_top_k_ends_far_below_the_maximum(V, bulk, T):
    """One likely id and a bulk over 36 temperatures (and 17) below it: the ids of top-k beyond
    the first have next to no weight, but which they are decides. A drafted id of the target's
    last rank that the drafter does not keep is accepted whatever the uniform, the id of the
    next rank is rejected whatever the uniform; one that both rows hold at equal logits, but
    only the target keeps, is accepted. No uniform lies near a ratio: they are 0 or infinite,
    against 0.5 and 0.999."""
    g, k = 4, 3000
    r = np.random.default_rng(V + int(4 * T))
    far = max(36.0 * T, 17.0)
    depth = {"one value": lambda: np.zeros(V), "few values": lambda: r.integers(0, 3, V) * 0.5,
             "spread": lambda: 20 * r.random(V)}[bulk]
    B = 3
    z = np.zeros((B, g + 1, V), dtype=np.float32)
    zq = np.zeros((B, g, V), dtype=np.float32)
    x = np.zeros((B, g), dtype=np.int32)
    for b in range(B):
        for j in range(g + 1):
            z[b, j] = -far - depth()
            z[b, j, 7] = 0.0
        for j in range(g):
            zq[b, j] = z[b, j] if b == 2 else -far - depth()[::-1]
            zq[b, j, 7] = 0.0
    zqd = torch.from_numpy(zq).to(torch.bfloat16).double().numpy()
    rank = lambda a: np.lexsort((np.arange(V), -a.astype(np.float64)))
    ua = np.full((B, g), 0.999, dtype=np.float32)
    for b in range(B):
        for j in range(g):
            order, mine = rank(z[b, j]), rank(zqd[b, j])
            kept_q = np.zeros(V, dtype=bool)
            kept_q[mine[:k]] = True
            inside = [i for i in order[:k] if not kept_q[i]]
            outside = [i for i in order[k:] if not kept_q[i]]
            x[b, j] = inside[-1] if b == 0 and inside else 7
            if b == 1 and j == 2:
                x[b, j] = outside[0]
                ua[b, j] = 0.5
            if b == 2 and j < 3 and inside:
                x[b, j] = inside[0]
    x[0, g - 1] = rank(z[0, g - 1])[k]
    settings = [(T, k, 1.0, 0.0)] * B
    for b in range(B):                      # id 7 is certain in both rows
        for j in range(g):
            w = F.filtered(z[b, j].astype(np.float64), *settings[b])[0]
            assert w[7] == 1.0 and w.sum() < 1 + 1e-6
    got, want = accept(z, zq, x, ua, r.random((B, g + 1), dtype=np.float32), settings)
    assert want[0][1] == 2                  # the id past the last rank is rejected
    assert got[0] == want[0]
    # The residuals of the rejected positions: id 7 has none or 1e-12, every other id at most its
    # p' <= e^-36 = 2.4e-16, about half of the unit 2^-51 = 4.4e-16 that residuals are summed in.
    # Which of those ids is drawn is therefore left open, not that the target keeps it.
    for b in range(B):
        if want[0][b] == g:
            assert got[1][b] == want[1][b] == 7
        else:
            assert F.filtered(z[b, want[0][b]].astype(np.float64), *settings[b])[0][got[1][b]] > 0


@pytest.mark.parametrize("V,B", [(4001, 2), (24001, 2)])
def test_min_p_under_the_binned_range(V, B):
    """A min-p border more than 33 temperatures below the maximum, many ids there: the row's
    weight is that of its 1400 equal likely ids, p' = 1 / 1400, against a q' of 1 / 700 (the
    acceptance probability is a half, to 1e-11): accepted at 0.4, rejected at 0.6."""
    g, n = 3, 1400
    r = np.random.default_rng(V)
    low = -33.0 + 0.5 * 33.0 / 2048          # the lowest bin's middle
    z = np.full((B, g + 1, V), -60.0, dtype=np.float32)
    zq = np.full((B, g, V), -60.0, dtype=np.float32)
    x = np.zeros((B, g), dtype=np.int32)
    for b in range(B):
        for j in range(g + 1):
            ids = r.permutation(V)
            z[b, j, ids[:n]] = 0.0
            z[b, j, ids[n:2 * n]] = low
            if j < g:
                zq[b, j, ids[:n // 2]] = 0.0
                x[b, j] = ids[r.integers(n // 2)]
    ua = np.full((B, g), 0.4, dtype=np.float32)
    for b in range(B):
        ua[b, 1 + b % 2] = 0.6
    settings = [(1.0, 0, 1.0, float(np.float32(1e-15)))] * B
    # the residual's 700 equal ids: uniforms in the middle of one's share
    ur = ((np.floor(r.random((B, g + 1)) * 600) + 0.5) / 700).astype(np.float32)
    got, want = accept(z, zq, x, ua, ur, settings)
    assert want[0] == [1 + b % 2 for b in range(B)]
    assert got[0] == want[0]
    assert got[1] == want[1]
