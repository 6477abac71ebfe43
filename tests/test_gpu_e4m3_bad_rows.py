"""The 8-bit paged cache where a row with an infinity or NaN comes and is taken back."""
import numpy as np
import pytest
import torch

from oracle import e4m3
from tests._e4m3 import D, Pool, check_attention, ints

pytestmark = pytest.mark.gpu


def _same_bits(p, state):
    p.same(state)
    got = p.host()
    for i in (1, 3):
        assert np.array_equal(got[i].view(np.uint32), state[i].view(np.uint32))


@pytest.mark.parametrize("cached", [(0, 1, 15, 16), (3, 17, 30, 28)])
@pytest.mark.parametrize("odd_scales", [False, True])
def test_a_rejected_draft_leaves_no_trace(cached, odd_scales):
    """Drafts with bad rows in some heads, K or V, then rows in their place: bit for bit as the
    model has it, and where scales are powers of two as without the bad rows."""
    p = Pool(4, 8, 2, 64, seed=sum(cached))
    p.fill(cached)
    if odd_scales:
        p.ks.mul_(1.5), p.vs.mul_(1.25)
    state, before, kvc = p.host(), p.host(), p.kvc

    def store(k, v, c, to):
        n = len(k) // 4
        kvc.check(kvc.kvc_append_packed(p.h, 0, k, v, ints([n * b for b in range(5)]), ints(c), 4 * n))
        for b in range(4):
            for i, x in ((0, k), (2, v)):
                for s in to:
                    e4m3.append(s[i], s[i + 1], p.order[b], c[b], x[n * b:n * b + n].float().cpu().numpy())

    k, v = p.normal(20, 2, D, tag="draft k"), p.normal(20, 2, D, tag="draft v")
    k[0, 0, 5], k[7, 1, 127], v[6, 0, 0], v[12, 1, 77], k[19] = np.inf, np.nan, -np.inf, np.inf, np.nan
    store(k, v, cached, [state])
    _same_bits(p, state)
    assert np.isnan(state[1]).any() and np.isnan(state[3]).any()
    # the first bad rows are 0, 1, 2 and 4 of the drafts
    for b, good in enumerate((0, 1, 2, 4)):
        for i, x in ((0, k), (2, v)):
            e4m3.append(before[i], before[i + 1], p.order[b], cached[b], x[5 * b:5 * b + good].float().cpu().numpy())
    c = [a + good for a, good in zip(cached, (0, 1, 2, 4))]
    k2, v2 = p.normal(8, 2, D, tag="next k"), p.normal(8, 2, D, tag="next v")
    store(k2, v2, c, [state, before])
    _same_bits(p, state)
    rows = [a + 2 for a in c]
    for b in range(4):
        blocks = p.order[b, :-(-rows[b] // 16)]
        assert np.isfinite(state[1][blocks]).all() and np.isfinite(state[3][blocks]).all()
        if not odd_scales:
            for i in (0, 2):
                assert torch.equal(e4m3.gather(state[i], state[i + 1], p.order[b], rows[b]), e4m3.gather(before[i], before[i + 1], p.order[b], rows[b]))
    q = p.normal(4, 8, D, tag="q")
    out = torch.zeros_like(q)
    kvc.check(kvc.kvc_packed_attn(p.h, 0, q, None, ints([r - 1 for r in rows]), 4, 0, out))
    check_attention(p, q, out, [0, 1, 2, 3, 4], [r - 1 for r in rows])
    assert p.error() == 0 and p.intact()


def test_rows_behind_a_bad_one_are_lost():
    """They read as NaN, and so does a block whose NaN keeps nothing, until its first row is stored."""
    p = Pool(1, 8, 2, 64, seed=3)
    kvc, state = p.kvc, p.host()
    x = p.normal(10, 2, D, tag="x")
    x[4, 1, 3] = np.nan
    q = p.normal(1, 8, D, tag="q")
    out = torch.zeros_like(q)

    def store(part, at):
        kvc.check(kvc.kvc_append_packed(p.h, 0, part, part, ints([0, len(part)]), ints([at]), len(part)))
        for i in (0, 2):
            e4m3.append(state[i], state[i + 1], p.order[0], at, part.float().cpu().numpy())
        _same_bits(p, state)
        kvc.check(kvc.kvc_packed_attn(p.h, 0, q, None, ints([at + len(part) - 1]), 1, 0, out))
        return out[0, :4].isfinite().all().item(), out[0, 4:].isfinite().all().item()
    assert store(x[:10], 0) == (True, False)
    assert store(x[:3], 10) == (True, False)
    assert store(x[5:7], 5) == (True, False)
    assert store(x[5:6], 4) == (True, True)
    p.ks[0, int(p.order[0, 0])] = state[1][int(p.order[0, 0])] = np.nan
    assert store(x[:2], 5) == (False, False)
    assert store(x[:1], 0) == (True, True)
    assert p.error() == 0 and p.intact()


@pytest.mark.parametrize("G, n", [(8, (1503, 1300)), (2, (70, 33))])
def test_bad_rows_in_prompts(G, n):
    """Blocks of long and short prompts, rotated: bad rows in some of them, the others as ever."""
    p = Pool(2, G, G, 1600, seed=G)
    cached = (37, 16)
    p.fill(cached)
    state, kvc, total = p.host(), p.kvc, sum(n)
    x = p.normal(total, 3 * G, D, tag="qkv")
    rng = np.random.default_rng(G)
    for r in rng.integers(0, total, 12):
        x[int(r), int(rng.integers(G, 3 * G)), int(rng.integers(D))] = float(rng.choice([np.inf, -np.inf, np.nan]))
    a = rng.uniform(-40, 40, (1600, 32))
    cs = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
    csd, q_out = torch.from_numpy(cs).cuda(), torch.zeros(total, G, D, dtype=torch.bfloat16, device="cuda")
    rope = kvc.make_rope(csd, 1600, 64, True)
    flat, s = x.view(total, -1), 3 * G * D
    kvc.check(kvc.kvc_append_rope(p.h, 0, rope, flat, s, flat[:, G * D:], s, flat[:, 2 * G * D:], s, ints([0, n[0], total]), ints(cached), total, q_out, None))
    host = x.float().cpu().numpy()
    with np.errstate(invalid="ignore"):
        k = e4m3.rotate(host[:, G:2 * G], cs, [c + i for c, m in zip(cached, n) for i in range(m)], 64, True)
    for b, lo, hi in ((0, 0, n[0]), (1, n[0], total)):
        e4m3.append(state[0], state[1], p.order[b], cached[b], k[lo:hi])
        e4m3.append(state[2], state[3], p.order[b], cached[b], host[lo:hi, 2 * G:])
    _same_bits(p, state)
    assert np.isnan(state[1]).any() and np.isnan(state[3]).any()
    assert p.error() == 0 and p.intact()


def test_bad_rows_in_dense_appends():
    """kvc_append's layout, and kvc_decode_step: a token's bad row, then the token again."""
    p = Pool(3, 4, 2, 96, "fp16", seed=11)
    kvc, cached = p.kvc, [20, 0, 7]
    p.fill(cached)
    state = p.host()
    k, v = p.normal(3, 2, 40, D, tag="k"), p.normal(3, 2, 40, D, tag="v")
    k[0, 1, 7, 3], v[2, 0, 39, 0], v[1, 1, 0, 5] = np.nan, np.inf, -np.inf
    kvc.check(kvc.kvc_append(p.h, 0, k, v, ints(cached), 40))
    for b, c in enumerate(cached):
        for i, y in ((0, k), (2, v)):
            e4m3.append(state[i], state[i + 1], p.order[b], c, y[b].transpose(0, 1).float().cpu().numpy())
    _same_bits(p, state)
    # sequence 2's last token again, through the step; the others on from rows that are good
    at = [26, 0, 46]
    k1, v1, q = p.normal(3, 2, 1, D, tag="k1"), p.normal(3, 2, 1, D, tag="v1"), p.normal(3, 4, D, tag="q")
    out = torch.zeros_like(q)
    kvc.check(kvc.kvc_decode_step(p.h, 0, q, k1, v1, ints([a + 1 for a in at]), 0, out))
    for b, c in enumerate(at):
        for i, y in ((0, k1), (2, v1)):
            e4m3.append(state[i], state[i + 1], p.order[b], c, y[b].transpose(0, 1).float().cpu().numpy())
    _same_bits(p, state)
    check_attention(p, q, out, [0, 1, 2, 3], at)
    assert p.error() == 0 and p.intact()
