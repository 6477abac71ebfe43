"""One key with most of the weight over a long flat tail: what the many small
probabilities add up to is as exact as the rest of the sum."""
import math

import numpy as np
import pytest
import torch

from oracle import e4m3
from tests._e4m3 import D, DT, Pool, cumulative, guarded, ints

pytestmark = pytest.mark.gpu

V_SCALE = 2.0 ** -8


def _fill(p, rows, sink, flat):
    """Sequence 0: keys whose scores are exact in fp32 (small whole numbers in nine
    columns), one of them told apart by column 0; values around 1, the sink's near 0."""
    gen = torch.Generator(device="cuda").manual_seed(p.seed + 1)
    room = -(-rows // 16) * 16
    K, V = torch.zeros(2, room, p.G, D, device="cuda")
    if not flat:
        K[:, :, 1:9] = torch.randint(-2, 3, (room, p.G, 8), generator=gen, device="cuda").float()
    K[sink, :, :9] = 0
    K[sink, :, 0] = 1
    V[:] = (1 + 0.25 * torch.randn(1 if flat else room, p.G, D, generator=gen, device="cuda")).clamp(0, 1.75)
    V[sink] = 0.01 * torch.randn(p.G, D, generator=gen, device="cuda")
    blocks = torch.from_numpy(p.order[0, :room // 16]).long().cuda()
    for X, scales, y, s in ((p.K, p.ks, K, 1.0), (p.V, p.vs, V, V_SCALE)):
        codes = (y / s).to(torch.float8_e4m3fn).view(torch.uint8)
        X[0, blocks] = codes.view(-1, 16, p.G, D).transpose(1, 2)
        scales[0, blocks] = s
    at = torch.from_numpy(p.order[0]).long().cuda()
    values = torch.from_numpy(e4m3.VALUES).cuda()
    wide = lambda X, s: (values[X[0, at].long()] * s[0, at][..., None, None].double()).transpose(0, 1).reshape(p.G, -1, D)[:, :rows]  # noqa: E731
    return wide(p.K, p.ks), wide(p.V, p.vs)


def _queries(p, n, k, sink, share):
    """[n, H, D]: the sink's score is what gives it `share` of the weight of all rows."""
    rng = np.random.default_rng(p.seed + 2)
    q = np.zeros((n, p.H, D))
    q[:, :, 1:9] = rng.choice([-2, -1, -0.5, 0.5, 1, 2], (n, p.H, 8))
    q = torch.from_numpy(q).cuda()
    s = torch.einsum("nhd,hjd->nhj", q, k.repeat_interleave(p.H // p.G, 0)) / math.sqrt(D)
    s[:, :, sink] = -math.inf
    q[:, :, 0] = (torch.logsumexp(s, 2) + math.log(share / (1 - share))) * math.sqrt(D)
    return q.to(DT[p.dtype])


# H, G, new tokens: 1, 4, 32 and 64 query rows per KV head, several of them drafted tokens, query rows on M
FORMS = [(1, 1, 1), (8, 2, 1), (32, 8, 1), (8, 2, 3), (32, 1, 1), (64, 1, 1), (12, 2, 10), (32, 8, 200)]


@pytest.mark.parametrize("H, G, n", FORMS)
@pytest.mark.parametrize("share, rows, where", [(0.9, 32768, "first"), (0.97, 16384, "first"), (0.97, 8192, "middle"), (0.9, 16384, "last"), (0.5, 16384, "flat")])
@pytest.mark.parametrize("splits", [1, 0])
def test_sink_and_tail(H, G, n, share, rows, where, splits):
    _check(H, G, n, share, rows, where, splits, 2.0 ** -29)


@pytest.mark.parametrize("H, G, n", FORMS)
@pytest.mark.parametrize("share, rows", [(0.97, 300), (0.99, 1024), (0.97, 2047), (0.97, 4096)])
def test_sink_and_short_tail(H, G, n, share, rows):
    """Fewer rows: the largest probability is 2^0 in those units below 1,024 of them, and all
    that they lose 2^-15 of it."""
    _check(H, G, min(n, 60), share, rows, "first", 1, 2.0 ** -15 / rows)


def _check(H, G, n, share, rows, where, splits, least):
    """An error of a probability: 2^-15 of it as four e4m3 values (2^-11 as an fp16 value, with
    query rows on M), with 2^-20 for the exponent (it is below 2^5) and the exponential, or `least` of the largest probability (times scale) that
    the row meets, 2^-25 in units in which that is 2^4 or more; sums over the keys round once per instruction, of 16
    keys at least.  The scores are exact."""
    n = min(n, 10) if rows > 20000 else n
    p = Pool(1, H, G, -(-rows // 16) * 16, "fp16" if H != 8 else "bf16", seed=H + n)
    sink = {"first": 0, "middle": rows // 2 + 5, "last": rows - n, "flat": 3}[where]
    k, v = _fill(p, rows, sink, where == "flat")
    q = _queries(p, n, k, sink, share)
    buf, out = guarded(torch.full((n, H, D), 7.0, dtype=DT[p.dtype], device="cuda"))
    p.kvc.check(p.kvc.kvc_set_num_splits(p.h, splits))
    p.kvc.check(p.kvc.kvc_packed_attn(p.h, 0, q, ints(cumulative([n])), ints([rows - n]), n, 0, out))
    assert p.error() == 0 and p.intact() and buf.canaries_intact()
    g = H // G
    s = torch.einsum("nhd,hjd->nhj", q.double(), k.repeat_interleave(g, 0)) / math.sqrt(D)
    s.masked_fill_(torch.arange(rows, device="cuda") > rows - n + torch.arange(n, device="cuda")[:, None, None], -math.inf)
    prob = torch.softmax(s, 2)
    assert float(prob[-1, :, sink].min()) > 0.8 * share
    v = v.repeat_interleave(g, 0)
    ref, mass = torch.einsum("nhj,hjd->nhd", prob, v), torch.einsum("nhj,hjd->nhd", prob, v.abs())
    err = ((2.0 ** -11 if n == 200 else 2.0 ** -15) + 2.0 ** -20 + (rows / 16 + 8) * 2.0 ** -23) * mass + rows * least * 448 * V_SCALE * prob.amax(2)[..., None]
    eps = torch.finfo(DT[p.dtype]).eps
    tol = err + eps / 2 * (ref.abs() + err) + (2.0 ** -25 if p.dtype == "fp16" else 0.0)
    worst = ((out.double() - ref).abs() / tol).amax()
    assert float(worst) <= 1, f"{float(worst):.2f} x tolerance; off by {float(((out.double() - ref).abs() / ref.abs()).amax()):.2e} of the result at most"
