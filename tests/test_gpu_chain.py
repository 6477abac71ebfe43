"""Calls that change a paged cache's table and calls that read it, one behind
the other in one captured graph with nothing between them: each sees what the
one before it left."""
import numpy as np
import pytest
import torch

from oracle import rows
from tests import _rows
from tests.test_gpu_pages import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("store", ["append", "commit"])
def test_attention_between_page_operations(store):
    """24 times over in one graph: attention, fork, reserve, rows stored,
    attention, a decode step, free.  Sequences 0-3 move on by one with every
    fork and 4-7 become copies of them, so that a table line of a step before
    leads to another sequence's rows."""
    B, H, G, D, n0, new, T, steps = 8, 4, 2, 64, 37, 5, 3, 24
    p = Pool(L=1, B=B, G=G, D=D, per=4, blocks=60, H=H, seed=5)
    k = p.kvc
    gen = torch.Generator(device="cuda").manual_seed(6)
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    p.reserve([0] * B, [n0] * B)
    p.check()
    parent = [1, 2, 3, 0, 1, 2, 3, 0]
    dev = {x: _rows.ints(v) for x, v in dict(parent=parent, n0=[n0] * B, n1=[n0 + new] * B, n2=[n0 + new + 1] * B,
                                             cu=np.arange(B + 1) * new, path=np.tile(np.arange(new), (B, 1)),
                                             taken=[new] * B).items()}
    q, kt, vt = draw(B, H, T, D), draw(B, G, T, D), draw(B, G, T, D)
    q1, k1, v1 = draw(B, H, D), draw(B, G, 1, D), draw(B, G, 1, D)
    kn, vn = draw(B, G, new, D), draw(B, G, new, D)          # row i of sequence b at n0 + i
    packed = [x.transpose(1, 2).reshape(B * new, G, D).contiguous() for x in (kn, vn)]
    outs = [(torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q1)) for _ in range(steps)]
    ws = torch.empty(k.kvc_rows_workspace_bytes(p.cfg), dtype=torch.uint8, device="cuda")
    state = (p.h, p.table, p.refs)

    def step(i, s):
        before, after, decoded = outs[i]
        attn = lambda n, o: k.kvc_tree_attn(p.h, 0, q, kt, vt, n, None, None, T, n0 + new, ws, ws.numel(), o, s)  # noqa: E731
        assert attn(dev["n0"], before) == 0
        assert k.kvc_pages_fork(*state, dev["parent"], s) == 0
        assert k.kvc_pages_reserve(*state, dev["n0"], dev["n2"], p.scratch.data, p.scratch.nbytes, s) == 0
        if store == "append":
            assert k.kvc_append_packed(p.h, 0, *packed, dev["cu"], dev["n0"], B * new, s) == 0
        else:
            assert k.kvc_tree_commit(p.h, 0, 1, kn, vn, dev["n0"], dev["path"], dev["taken"], new, new, s) == 0
        assert attn(dev["n1"], after) == 0
        assert k.kvc_decode_step(p.h, 0, q1, k1, v1, dev["n2"], n0 + new + 1, decoded, s) == 0
        assert k.kvc_pages_free(*state, dev["n0"], s) == 0

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for i in range(steps):
                step(i, side)
    torch.cuda.synchronize()
    chain = torch.ones(T, T, dtype=torch.bool).tril()
    one = torch.ones(1, 1, dtype=torch.bool)
    hist = [[X[0, p.model.table[b]].transpose(0, 1).reshape(G, -1, D)[:, :n0].clone() for X in (p.K, p.V)] for b in range(B)]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for i in range(steps):
            before, after, decoded = outs[i]
            for b in range(B):
                _rows.close(before[b], *rows.attend(q[b], *hist[b], kt[b], vt[b], chain), "bf16", D, n0 + T, f"step {i}, before")
            hist = [hist[x] for x in parent]
            p.model.fork(parent)
            p._moved(p.model.reserve([n0] * B, [n0 + new + 1] * B))
            for b in range(B):
                full = [torch.cat([h, x[b]], 1) for h, x in zip(hist[b], (kn, vn))]
                _rows.close(after[b], *rows.attend(q[b], *full, kt[b], vt[b], chain), "bf16", D, n0 + new + T, f"step {i}, after")
                ref = rows.attend(q1[b][:, None], *full, k1[b], v1[b], one)[0]
                assert (decoded[b].double() - ref[:, 0]).abs().max() <= 2e-2, f"step {i}, decoded"
                for j in range(n0, n0 + new + 1):
                    at = (0, p.model.table[b][j // 16], slice(None), j % 16)
                    for X, x, x1 in ((p.k_want, kn, k1), (p.v_want, vn, v1)):
                        X[at] = x[b, :, j - n0] if j < n0 + new else x1[b, :, 0]
            p.model.free([n0] * B)
        p.check()
