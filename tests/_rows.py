"""Shared by the GPU tests of the prompt, tree and page calls: caches with
cached rows of given lengths, packed and drafted rows, and the comparison with
oracle.rows."""
import numpy as np
import torch

from oracle import rows
from static_kv_cache_gb300 import synth
from tests import _gpu


def guarded(values):
    """A copy of a tensor between canaries."""
    buf = _gpu.Guarded(max(16, values.numel() * values.element_size()))
    view = buf.data[:values.numel() * values.element_size()].view(values.dtype).view(values.shape)
    view.copy_(values)
    return buf, view


class Cache:
    """A contiguous or paged cache whose rows hold poison except for the first
    ``cached[b]`` of every sequence."""

    def __init__(self, dtype, L, B, H, G, D, T, paged=False, spare=3, seed=0, device="cuda"):
        from static_kv_cache_gb300 import kvc
        self.kvc, self.dtype, self.tdt = kvc, dtype, synth.DTYPES[dtype]
        self.act = synth.ACT_DTYPE[dtype]
        self.L, self.B, self.H, self.G, self.D, self.T, self.paged, self.seed = L, B, H, G, D, T, paged, seed
        self.cfg = kvc.make_config(L, B, H, G, D, T, dtype)
        self.ws = _gpu.Guarded(kvc.kvc_workspace_bytes(self.cfg))
        if paged:
            mb = T // 16
            self.blocks = B * mb + spare
            shape = (L, self.blocks, G, 16, D)
        else:
            shape = (L, B, G, T, D)
        nbytes = int(np.prod(shape)) * synth.ELEM_BYTES[dtype]
        self.bufs = [_gpu.Guarded(nbytes), _gpu.Guarded(nbytes), self.ws]
        self.K, self.V = (b.view(self.tdt, shape) for b in self.bufs[:2])
        if dtype == "int8":
            self.K.fill_(99), self.V.fill_(99)
            self.sbufs = [_gpu.Guarded(L * B * G * T * 4) for _ in range(2)]
            self.ks, self.vs = (b.view(torch.float32, (L, B, G, T)) for b in self.sbufs)
            self.ks.fill_(-3.0), self.vs.fill_(-3.0)
            self.bufs += self.sbufs
            st, self.h = kvc.kvc_alloc_scaled(self.cfg, self.bufs[0].ptr(), self.bufs[1].ptr(), self.sbufs[0].ptr(),
                                              self.sbufs[1].ptr(), self.ws.ptr(), self.ws.nbytes)
        else:
            synth.poison_(self.K, dtype)
            synth.poison_(self.V, dtype)
            if paged:
                order = np.random.default_rng(seed).permutation(self.blocks)[:B * mb].reshape(B, mb).astype(np.int32)
                self.tbuf, self.table = guarded(torch.from_numpy(order).cuda())
                self.bufs.append(self.tbuf)
                st, self.h = kvc.kvc_alloc_paged(self.cfg, self.bufs[0].ptr(), self.bufs[1].ptr(), self.blocks,
                                                 self.tbuf.ptr(), self.ws.ptr(), self.ws.nbytes)
            else:
                st, self.h = kvc.kvc_alloc(self.cfg, self.bufs[0].ptr(), self.bufs[1].ptr(), self.ws.ptr(), self.ws.nbytes)
        kvc.check(st, "alloc")
        self.scratch = _gpu.Guarded(kvc.kvc_rows_workspace_bytes(self.cfg))
        self.bufs.append(self.scratch)

    def __del__(self):
        if getattr(self, "h", None):
            self.kvc.kvc_free(self.h)

    def draw(self, *shape, tag=0):
        return synth.normal(shape, self.act, synth.sub_seed(self.seed, "rows", tag, shape), device="cuda")

    def at(self, X, layer, b, rows_):
        """Positions ``rows_`` of sequence b as an index into X: [G, n, D]."""
        i = torch.as_tensor(rows_, device="cuda", dtype=torch.long)
        if self.paged:
            return X[layer][self.table[b, i // 16].long(), :, i % 16].transpose(0, 1)
        return X[layer, b][:, i]

    def put(self, X, layer, b, rows_, values):
        i = torch.as_tensor(rows_, device="cuda", dtype=torch.long)
        if self.paged:
            X[layer][self.table[b, i // 16].long(), :, i % 16] = values.transpose(0, 1)
        else:
            X[layer, b][:, i] = values

    def fill(self, layer, cached):
        for b, n in enumerate(cached):
            if n:
                self.put(self.K, layer, b, range(n), self.draw(self.G, n, self.D, tag=("k", layer, b)))
                self.put(self.V, layer, b, range(n), self.draw(self.G, n, self.D, tag=("v", layer, b)))

    def error(self):
        return self.kvc.kvc_get_error(self.h, None)

    def intact(self):
        return all(b.canaries_intact() for b in self.bufs)


def ints(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def tree(T, seed, chain=False):
    """A random tree as a bool [T, T]: row t marks t and the tokens above it."""
    rng = np.random.default_rng(seed)
    seen = np.zeros((T, T), bool)
    for t in range(T):
        up = t - 1 if chain else int(rng.integers(-1, t)) if t else -1
        if up >= 0:
            seen[t] = seen[up]
        seen[t, t] = True
    return torch.from_numpy(seen)


def words(seen):
    """bool [B, T, T] as the call's 32-bit words."""
    B, T, _ = seen.shape
    W = -(-T // 32)
    bits = np.zeros((B, T, W * 32), np.uint64)
    bits[:, :, :T] = seen.numpy()
    return torch.from_numpy((bits.reshape(B, T, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)).cuda()


def close(got, out, mass, reach, dtype, D, keys, what=""):
    """Element by element within the derived tolerance; infinities and NaN where
    the definition has them, and nowhere else."""
    tol = rows.tolerance(out, mass, reach, dtype, D, keys)
    err = (got.double() - out).abs()
    fine = torch.isfinite(out)
    same = (got.double() == out) | (got.isnan() & out.isnan())
    bad = torch.where(fine, ~(err <= tol), ~same)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).max()):.2f} x tolerance, got {got[bad][:4].tolist()}, want {out[bad][:4].tolist()}"
