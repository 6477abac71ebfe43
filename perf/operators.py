"""Serving operators around the static KV cache, measured case by case.

Five operators, each a step in the life of a batch of sequences whose keys and
values sit in a contiguous or a paged cache:

  prompt   causal attention of prompts of different lengths packed one behind
           the other, over their own rows and, where a prefix is cached
           already, over the cache             (kvc_prompt_attn)
  ingest   the packed prompts' K and V rows into the cache
                                               (kvc_append_packed)
  tree     attention of a tree of drafted tokens over the cache and over the
           drafted tokens on each token's own path
                                               (kvc_tree_attn)
  commit   the accepted path's K and V rows into the cache, every layer
                                               (kvc_tree_commit)
  pages    the pages of a paged cache: forked between beams and made writable
           (kvc_pages_fork, kvc_pages_reserve), freed and compacted
           (kvc_pages_free, kvc_pages_compact)

``own = False`` computes them in elementary torch operations, ``own = True``
calls the library.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # A chat server's short turns: 24 prompts of a few to 300 tokens on the
        # 12-over-2-heads shape, nothing cached before.  Latency counts.
        {"name": "prompt_short", "op": "prompt", "dtype": "fp16", "batch": 24, "heads": 12, "kv_heads": 2, "d_head": 128,
         "shortest": 1, "longest": 300, "prefix": 0, "paged": False, "mix": 1},
        # A batch of ordinary documents of mixed lengths on the Llama-3-8B heads,
        # each continuing a cached prefix of up to 1500 rows (a shared system
        # prompt, the turns before) that sits in pages.
        {"name": "prompt_over_prefix", "op": "prompt", "dtype": "bf16", "batch": 8, "heads": 32, "kv_heads": 8, "d_head": 128,
         "shortest": 64, "longest": 2048, "prefix": 1500, "paged": True, "mix": 2},
        # One long document: the largest, bound by the tensor cores.
        {"name": "prompt_long", "op": "prompt", "dtype": "bf16", "batch": 1, "heads": 32, "kv_heads": 8, "d_head": 128,
         "shortest": 16384, "longest": 16384, "prefix": 0, "paged": False, "mix": 3},
        # The short turns' rows go into a contiguous cache.
        {"name": "ingest_short", "op": "ingest", "dtype": "fp16", "batch": 24, "heads": 12, "kv_heads": 2, "d_head": 128,
         "shortest": 1, "longest": 300, "prefix": 0, "paged": False, "mix": 1},
        # The documents' rows behind their prefixes, through the block table.
        {"name": "ingest_paged", "op": "ingest", "dtype": "bf16", "batch": 16, "heads": 32, "kv_heads": 8, "d_head": 128,
         "shortest": 64, "longest": 8000, "prefix": 190, "paged": True, "mix": 4},
        # One user, a small tree of drafts over a short context: latency.
        {"name": "tree_one_user", "op": "tree", "dtype": "bf16", "batch": 1, "heads": 32, "kv_heads": 8, "d_head": 128,
         "nodes": 13, "shortest": 700, "longest": 700, "paged": False, "mix": 5},
        # A ragged batch in pages, 32 drafted tokens each (some trees pruned).
        {"name": "tree_batch_paged", "op": "tree", "dtype": "bf16", "batch": 16, "heads": 32, "kv_heads": 8, "d_head": 128,
         "nodes": 32, "shortest": 1024, "longest": 8192, "paged": True, "mix": 6},
        # Long contexts without grouped heads: bound by the cache's bytes.
        {"name": "tree_long_mha", "op": "tree", "dtype": "fp16", "batch": 4, "heads": 64, "kv_heads": 64, "d_head": 128,
         "nodes": 60, "shortest": 20000, "longest": 32000, "paged": False, "mix": 7},
        # One user's accepted path, every layer of the Llama-3-8B shape.
        {"name": "commit_one_user", "op": "commit", "dtype": "bf16", "batch": 1, "layers": 32, "heads": 32, "kv_heads": 8,
         "d_head": 128, "nodes": 13, "longest": 700, "paged": False, "mix": 8},
        # The same for a large batch in pages, deep paths accepted.
        {"name": "commit_batch_paged", "op": "commit", "dtype": "fp16", "batch": 64, "layers": 28, "heads": 12, "kv_heads": 2,
         "d_head": 128, "nodes": 48, "longest": 2000, "paged": True, "mix": 9},
        # A beam search's step: 16 requests of 4 beams take their parents' pages
        # and make the next token's row writable.
        {"name": "pages_beams", "op": "beams", "dtype": "bf16", "batch": 64, "group": 4, "layers": 8, "heads": 32, "kv_heads": 8,
         "d_head": 128, "longest": 1200, "spare": 300, "mix": 10},
        # A third of the sequences has ended, others were rewound; the pool is
        # compacted so that its tail can be given back.
        {"name": "pages_compact", "op": "evict", "dtype": "bf16", "batch": 32, "layers": 8, "heads": 32, "kv_heads": 8,
         "d_head": 128, "longest": 1500, "spare": 100, "mix": 11},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "ingest", "tree", "commit", "beams", "evict"])
    heads, kv_heads = rng.choice([(32, 8), (12, 2), (8, 2), (16, 16), (24, 8), (32, 1), (14, 2)])
    case = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "heads": heads, "kv_heads": kv_heads,
            "d_head": rng.choice([64, 128, 128]), "mix": rng.randrange(1 << 20)}
    if op in ("prompt", "ingest"):
        batch = _spread(rng, 1, 24)
        longest = _spread(rng, 4, max(8, 9000 // batch))
        case.update(batch=batch, shortest=rng.choice([0, 1, longest // 2]), longest=longest,
                    prefix=rng.choice([0, 0, _spread(rng, 1, 2000)]), paged=rng.random() < 0.5)
    elif op == "tree":
        longest = _spread(rng, 1, 16000)
        case.update(batch=_spread(rng, 1, 16), nodes=_spread(rng, 1, 128), shortest=rng.choice([0, longest // 2, longest]),
                    longest=longest, paged=rng.random() < 0.5)
    elif op == "commit":
        case.update(batch=_spread(rng, 1, 48), layers=_spread(rng, 1, 32), nodes=_spread(rng, 1, 100),
                    longest=_spread(rng, 1, 1500), paged=rng.random() < 0.5)
    elif op == "beams":
        group = rng.choice([1, 2, 3, 4, 8])
        case.update(batch=group * _spread(rng, 1, 12), group=group, layers=_spread(rng, 1, 8), longest=_spread(rng, 1, 1500),
                    spare=rng.randrange(100, 400))
    else:
        case.update(batch=_spread(rng, 1, 40), layers=_spread(rng, 1, 8), longest=_spread(rng, 16, 1500), spare=rng.randrange(0, 300))
    if case.get("paged") or op in ("beams", "evict"):
        case["heads"], case["kv_heads"] = rng.choice([(32, 8), (12, 2), (8, 2), (24, 8), (32, 1), (14, 2)])
    return case


# ------------------------------------------- what a case fixes besides sizes
def _mix(case, what):
    return np.random.RandomState([case["mix"], what])


def _lengths(case):
    """Prompt lengths (prompt, ingest), or cached rows of each sequence."""
    lo, hi = case.get("shortest", 1), case["longest"]
    n = _mix(case, 0).randint(lo, hi + 1, case["batch"])
    n[_mix(case, 1).randint(case["batch"])] = hi  # the longest is there
    return n


def _prefixes(case):
    if not case.get("prefix"):
        return np.zeros(case["batch"], int)
    return _mix(case, 2).randint(0, case["prefix"] + 1, case["batch"])


def _nodes(case):
    """Drafted tokens of each sequence; some trees are pruned."""
    n = np.full(case["batch"], case["nodes"])
    cut = _mix(case, 3).rand(case["batch"]) < 0.25
    n[cut] = _mix(case, 4).randint(0, case["nodes"] + 1, case["batch"])[cut]
    n[0] = case["nodes"]
    return n


def _accepted(case):
    return np.minimum(_mix(case, 5).randint(0, case["nodes"] + 1, case["batch"]), _nodes(case))


def _parents(case):
    """The beam that each beam continues: one of its own request's."""
    g, b = case["group"], case["batch"]
    return np.arange(b) // g * g + _mix(case, 6).randint(0, g, b)


def _kept(case):
    """Rows that each sequence keeps: a third ends, a third is rewound."""
    n = _lengths(case)
    what = _mix(case, 7).randint(0, 3, case["batch"])
    return np.where(what == 0, 0, np.where(what == 1, (n * _mix(case, 8).rand(case["batch"])).astype(int), n))


def _pages_of(rows):
    return -(-np.asarray(rows) // PAGE)


def _beam_lengths(case):
    """Beams of one request are equally long; the first half of their rows is their common prompt."""
    return np.repeat(_lengths({**case, "batch": case["batch"] // case["group"]}), case["group"])


# ------------------------------------------------------------------- inputs
def _ints(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def _ancestors(nodes, batch, gen):
    """Random trees: 0/1 [batch, nodes, nodes], row t marks t and the tokens above it."""
    parent = (torch.rand(batch, nodes, generator=gen) * (torch.arange(nodes) + 0.35)).floor().long() - 1
    seen = torch.zeros(batch, nodes, nodes, dtype=torch.bool)
    for t in range(nodes):  # a parent comes before its children
        up = parent[:, t]
        above = seen[torch.arange(batch), up.clamp(min=0)] & (up >= 0)[:, None]
        seen[:, t] = above
        seen[:, t, t] = True
    return seen


def _words(seen):
    """The same as 32-bit words, bit s of word w for token 32 w + s."""
    b, t, s = seen.shape
    w = -(-s // 32)
    bits = torch.zeros(b, t, w * 32, dtype=torch.int64)
    bits[:, :, :s] = seen
    words = (bits.view(b, t, w, 32) << torch.arange(32)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)
    cpu = torch.Generator().manual_seed(int(seed) * 7919 + 13)
    host = np.random.RandomState(int(seed) % (1 << 31))
    t, op = TYPES[case["dtype"]], case["op"]
    B, H, G, D = case["batch"], case["heads"], case["kv_heads"], case["d_head"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=t)

    s = {"case": case, "op": op, "B": B, "H": H, "G": G, "D": D, "L": case.get("layers", 1)}
    paged = case.get("paged", op in ("beams", "evict"))
    if op in ("prompt", "ingest"):
        n, c = _lengths(case), _prefixes(case)
        room = int((n + c).max()) if op == "ingest" else max(1, int(c.max()))
        cu = np.concatenate([[0], np.cumsum(n)])
        total = int(cu[-1])
        s.update(cu=_ints(cu), c=_ints(c), n=_ints(n), total=total, longest=int(n.max()), widest=int(c.max()),
                 prefix=bool(case["prefix"]), k=normal(total, G, D), v=normal(total, G, D))
        if op == "prompt":
            s.update(q=normal(total, H, D), out=torch.zeros(total, H, D, device="cuda", dtype=t))
        rows = n + c if op == "ingest" else c
    elif op in ("tree", "commit"):
        T, nodes = case["nodes"], _nodes(case)
        c = _lengths(case)
        s.update(T=T, c=_ints(c), n=_ints(nodes), widest=int(c.max()), k=normal(s["L"], B, G, T, D), v=normal(s["L"], B, G, T, D))
        room = int(c.max())
        rows = c
        if op == "tree":
            seen = _ancestors(T, B, cpu)
            s.update(seen=seen.cuda(), words=_words(seen).cuda(), q=normal(B, H, T, D),
                     out=torch.zeros(B, H, T, D, device="cuda", dtype=t), k=s["k"][0], v=s["v"][0])
        else:
            accepted = _accepted(case)
            # the accepted path: a rising choice of the drafted tokens
            order = np.argsort(host.rand(B, T) + (np.arange(T) >= nodes[:, None]), axis=1)
            path = np.sort(np.where(np.arange(T) < accepted[:, None], order, T), axis=1)
            s.update(path=_ints(np.where(path < T, path, 0)), accepted=_ints(accepted))
            room, rows = room + T, c + accepted
    elif op == "beams":
        n = _beam_lengths(case)
        s.update(n=_ints(n), grown=_ints(n + 1), parent=_ints(_parents(case)))
        room, rows = int(n.max()) + 1, n
    else:
        n = _lengths(case)
        s.update(n=_ints(n), kept=_ints(_kept(case)))
        room, rows = int(n.max()), n
    if not paged:
        s["K"], s["V"] = normal(s["L"], B, G, max(1, room), D), normal(s["L"], B, G, max(1, room), D)
        s["room"] = max(1, room)
    else:
        per = max(1, -(-room // PAGE))
        s["room"] = per * PAGE
        used = _pages_of(rows)
        spare = case.get("spare", 3)
        blocks = int(used.sum()) + spare
        order = host.permutation(blocks)
        table = np.full((B, per), -1)
        table[np.arange(per) < used[:, None]] = order[:int(used.sum())]
        if op == "beams":  # beams share the pages of their prompt
            first = np.arange(B) // case["group"] * case["group"]
            table = np.where(np.arange(per) < (rows // 2 // PAGE)[:, None], table[first], table)
        # one buffer for what a step changes: the table, then the counts
        book = np.concatenate([table.reshape(-1), np.zeros(-(B * per) % 4, int), np.zeros(blocks, int)])
        at = B * per + -(B * per) % 4
        book[at:] = np.bincount(table[table >= 0], minlength=blocks)
        s.update(blocks=blocks, book=_ints(book), book0=_ints(book), live=torch.zeros(1, dtype=torch.int32, device="cuda"))
        s["table"], s["refs"] = s["book"][:B * per].view(B, per), s["book"][at:]
        s["K"], s["V"] = normal(s["L"], blocks, G, PAGE, D), normal(s["L"], blocks, G, PAGE, D)
    if own:  # the handle that a program keeps
        s["handle"] = _Handle(s, paged)
    return s


class _Handle:
    """The library's handle over the state's cache, and the workspaces that go with it."""

    def __init__(self, s, paged):
        from static_kv_cache_gb300 import kvc
        self.kvc = kvc
        cfg = kvc.make_config(s["L"], s["B"], s["H"], s["G"], s["D"], s["room"], s["case"]["dtype"])
        self.ws = torch.empty(kvc.kvc_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
        if paged:
            st, self.h = kvc.kvc_alloc_paged(cfg, s["K"], s["V"], s["blocks"], s["table"], self.ws, self.ws.numel())
        else:
            st, self.h = kvc.kvc_alloc(cfg, s["K"], s["V"], self.ws, self.ws.numel())
        kvc.check(st, "alloc")
        need = kvc.kvc_rows_workspace_bytes(cfg) if s["op"] in ("prompt", "tree") else \
            kvc.kvc_pages_workspace_bytes(cfg, s["blocks"]) if s["op"] in ("beams", "evict") else 0
        self.scratch = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")

    def __del__(self):
        if getattr(self, "h", None):
            self.kvc.kvc_free(self.h)


# --------------------------------------------------------- one pass, either way
def run(s):
    if own:
        return _own(s)
    return {"prompt": _plain_prompt, "ingest": _plain_ingest, "tree": _plain_tree, "commit": _plain_commit,
            "beams": _plain_beams, "evict": _plain_evict}[s["op"]](s)


def _own(s):
    hd = s["handle"]
    kvc, h, ws, op = hd.kvc, hd.h, hd.scratch, s["op"]
    stream = torch.cuda.current_stream()
    if op == "prompt":
        kvc.check(kvc.kvc_prompt_attn(h, 0, s["q"], s["k"], s["v"], s["cu"], s["c"] if s["prefix"] else None, s["total"],
                                      ws, ws.numel(), s["out"], stream), "kvc_prompt_attn")
        return s["out"]
    if op == "ingest":
        kvc.check(kvc.kvc_append_packed(h, 0, s["k"], s["v"], s["cu"], s["c"] if s["prefix"] else None, s["total"], stream),
                  "kvc_append_packed")
        return s["K"], s["V"]
    if op == "tree":
        kvc.check(kvc.kvc_tree_attn(h, 0, s["q"], s["k"], s["v"], s["c"], s["n"], s["words"], s["T"], s["widest"],
                                    ws, ws.numel(), s["out"], stream), "kvc_tree_attn")
        return s["out"]
    if op == "commit":
        kvc.check(kvc.kvc_tree_commit(h, 0, s["L"], s["k"], s["v"], s["c"], s["path"], s["accepted"], s["T"], s["T"], stream),
                  "kvc_tree_commit")
        return s["K"], s["V"]
    s["book"].copy_(s["book0"])  # the same step again
    if op == "beams":
        kvc.check(kvc.kvc_pages_fork(h, s["table"], s["refs"], s["parent"], stream), "kvc_pages_fork")
        kvc.check(kvc.kvc_pages_reserve(h, s["table"], s["refs"], s["n"], s["grown"], ws, ws.numel(), stream), "kvc_pages_reserve")
        return s["table"], s["refs"], s["K"], s["V"]
    kvc.check(kvc.kvc_pages_free(h, s["table"], s["refs"], s["kept"], stream), "kvc_pages_free")
    kvc.check(kvc.kvc_pages_compact(h, s["table"], s["refs"], None, s["live"], ws, ws.numel(), stream), "kvc_pages_compact")
    return s["table"], s["refs"], s["live"], s["K"], s["V"]


# ------------------------------------------------------------ the plain forms
def _cached(s, X):
    """The first `widest` cached rows of every sequence, [B, G, widest, D] in 32 bits."""
    if "table" not in s:
        return X[0, :, :, :s["widest"]].float()
    pages = s["table"][:, :_pages_of(s["widest"])].clamp(min=0).long()
    rows = X[0][pages].transpose(1, 2)  # [B, G, pages, PAGE, D]
    return rows.reshape(s["B"], s["G"], -1, s["D"])[:, :, :s["widest"]].float()


def _attend(s, q, k, v, k_new, v_new, seen):
    """softmax(q K^T / sqrt(d)) V over the cached rows below c and the new rows
    that `seen` ([B, Q, N]) marks.  q [B, H, Q, D]; rows without a key give zeros."""
    B, G, D = s["B"], s["G"], s["D"]
    q = q.float().reshape(B, G, -1, D)
    past = torch.arange(k.shape[2], device="cuda")[None, None] < s["c"][:, None, None]
    seen = torch.cat([past.expand(-1, seen.shape[1], -1), seen], 2)
    x = q @ torch.cat([k, k_new.float()], 2).transpose(2, 3)
    x = x.view(B, G, -1, *seen.shape[1:]).mul_(1 / math.sqrt(D)).masked_fill_(~seen[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = x.sum(-1, keepdim=True)
    out = x.view(B, G, -1, seen.shape[2]) @ torch.cat([v, v_new.float()], 2)
    out = out / total.view(B, G, -1, 1).clamp(min=1e-30)
    return out.view(B, s["H"], -1, D)


def _plain_prompt(s):
    """Every prompt padded to the longest, attended, and packed again."""
    B, N, H, G, D = s["B"], s["longest"], s["H"], s["G"], s["D"]
    at = torch.arange(N, device="cuda")
    rows = s["cu"][:-1, None].long() + at
    real = at < s["n"][:, None]
    rows = torch.where(real, rows, 0)
    new = s["q"][rows].transpose(1, 2), s["k"][rows].transpose(1, 2), s["v"][rows].transpose(1, 2)
    seen = (at[None, :] <= at[:, None]) & real[:, None, :]
    o = _attend(s, new[0], _cached(s, s["K"]), _cached(s, s["V"]), new[1], new[2], seen)
    return o.transpose(1, 2)[real].to(s["q"].dtype)


def _plain_tree(s):
    nodes = torch.arange(s["T"], device="cuda")
    real = nodes < s["n"][:, None]
    seen = s["seen"] & real[:, None, :]
    o = _attend(s, s["q"], _cached(s, s["K"]), _cached(s, s["V"]), s["k"], s["v"], seen)
    return torch.where(real[:, None, :, None], o, 0).to(s["q"].dtype)


def _store(s, X, b, at, rows):
    """Cache row at[i] of sequence b[i], all layers: rows [L, i, G, D]."""
    if "table" in s:
        X.transpose(2, 3)[:, s["table"][b, at // PAGE].long(), at % PAGE] = rows
    else:
        X.transpose(2, 3)[:, b, at] = rows


def _plain_ingest(s):
    b = torch.repeat_interleave(torch.arange(s["B"], device="cuda"), s["n"].long(), output_size=s["total"])
    at = torch.arange(s["total"], device="cuda") - s["cu"][b].long() + s["c"][b].long()
    _store(s, s["K"], b, at, s["k"][None])
    _store(s, s["V"], b, at, s["v"][None])
    return s["K"], s["V"]


def _plain_commit(s):
    b, i = (torch.arange(s["T"], device="cuda") < s["accepted"][:, None]).nonzero(as_tuple=True)
    at, node = s["c"][b].long() + i, s["path"][b, i].long()
    _store(s, s["K"], b, at, s["k"].transpose(2, 3)[:, b, node])
    _store(s, s["V"], b, at, s["v"].transpose(2, 3)[:, b, node])
    return s["K"], s["V"]


def _count(s, table, by):
    """Adds `by` to the counts of every page that the table entries name."""
    s["refs"].index_add_(0, table.clamp(min=0).flatten(), (table >= 0).flatten().to(torch.int32) * by)


def _plain_beams(s):
    s["book"].copy_(s["book0"])
    table, refs = s["table"], s["refs"]
    # fork: every beam takes its parent's pages
    forked = torch.where(s["parent"][:, None] >= 0, table[s["parent"].clamp(min=0)], -1)
    _count(s, forked, 1)
    _count(s, table, -1)
    # reserve: a shared page that is about to be written is copied by all beams
    # but the last of those that hold it; pages past the end are added
    n, grown = s["n"], s["grown"]
    per = torch.arange(table.shape[1], device="cuda")
    part = (n % PAGE != 0) & (grown > n)
    page = torch.where(part, forked.gather(1, (n // PAGE).long().clamp(max=table.shape[1] - 1)[:, None])[:, 0], -1)
    before = ((page[:, None] == page[None, :]) & part[:, None] & part[None, :]).tril(-1).sum(1)
    split = part & (refs[page.clamp(min=0)] - before > 1)
    fresh = (per >= ((n + PAGE - 1) // PAGE)[:, None]) & (per < ((grown + PAGE - 1) // PAGE)[:, None])
    fresh |= split[:, None] & (per == (n // PAGE)[:, None])
    free = torch.argsort((refs != 0).to(torch.int8), stable=True).to(torch.int32)
    rank = fresh.flatten().cumsum(0).view(fresh.shape) - 1
    taken = torch.where(fresh, free[rank.clamp(min=0, max=len(free) - 1)], forked)
    refs.index_add_(0, page.clamp(min=0), -split.to(torch.int32))
    _count(s, torch.where(fresh, taken, -1), 1)
    table.copy_(taken)
    b = split.nonzero()[:, 0]
    old, new = page[b].long(), taken[b, (n[b] // PAGE).long()].long()
    live = (torch.arange(PAGE, device="cuda") < (n[b] % PAGE)[:, None])[None, :, None, :, None]
    s["K"][:, new] = torch.where(live, s["K"][:, old], s["K"][:, new])
    s["V"][:, new] = torch.where(live, s["V"][:, old], s["V"][:, new])
    return table, refs, s["K"], s["V"]


def _plain_evict(s):
    s["book"].copy_(s["book0"])
    table, refs = s["table"], s["refs"]
    # free: pages behind the rows that are kept
    gone = torch.arange(table.shape[1], device="cuda") >= ((s["kept"] + PAGE - 1) // PAGE)[:, None]
    _count(s, torch.where(gone, table, -1), -1)
    table.masked_fill_(gone, -1)
    # compact: the live pages at or above their number move, in order, to the free ones below it
    used, place = refs > 0, torch.arange(len(refs), device="cuda")
    live = used.sum()
    old, new = (used & (place >= live)).nonzero()[:, 0], (~used & (place < live)).nonzero()[:, 0]
    to = place.to(torch.int32)
    to[old] = new.to(torch.int32)
    s["K"][:, new], s["V"][:, new] = s["K"][:, old], s["V"][:, old]
    refs[new] = refs[old]
    refs[old] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0)], -1))
    s["live"].copy_(live)
    return table, refs, s["live"], s["K"], s["V"]


# ---------------------------------------------------- what a pass has to do
def work(case):
    B, H, G, D, op = case["batch"], case["heads"], case["kv_heads"], case["d_head"], case["op"]
    L, row = case.get("layers", 1), case["kv_heads"] * case["d_head"] * 2  # one token's keys (or values) of a layer
    if op == "prompt":
        n, c = _lengths(case).astype(float), _prefixes(case).astype(float)
        pairs = float((n * c + n * (n + 1) / 2).sum())
        return {"bytes": float(n.sum() * (2 * H * D * 2 + 2 * row) + (c * (n > 0)).sum() * 2 * row + 4 * (2 * B + 1)), "flops": 4.0 * D * H * pairs}
    if op == "tree":
        n, c = _nodes(case).astype(float), _lengths(case).astype(float)
        pairs = float((n * c + n * n / 4).sum())  # trees are sparse; a quarter stands for their marks
        return {"bytes": float(n.sum() * (2 * H * D * 2 + 2 * row) + (c * (n > 0)).sum() * 2 * row + 4 * n.sum() * -(-case["nodes"] // 32)),
                "flops": 4.0 * D * H * pairs}
    if op == "ingest":
        return {"bytes": float(_lengths(case).sum()) * 4 * row, "flops": 0}
    if op == "commit":
        return {"bytes": float(_accepted(case).sum()) * 4 * row * L + 8.0 * B, "flops": 0}
    if op == "beams":
        n, p = _beam_lengths(case), _parents(case)
        pages = float(_pages_of(n).sum())
        copies = np.array([n[b] % PAGE * int((p[b + 1:] == p[b]).any()) for b in range(B)]).sum()
        return {"bytes": float(copies) * 4 * row * L + pages * 16, "flops": 0}
    n, k = _lengths(case), _kept(case)
    total = _pages_of(n).sum() + case["spare"]
    live = float(_pages_of(k).sum())
    moved = live * (total - live) / total  # of the live pages, those that sit above their number
    return {"bytes": float(moved) * PAGE * 4 * row * L + 4.0 * (total + B * _pages_of(n.max())) + 8, "flops": 0}


# ------------------------------------------------------- the definition, exactly
def exact(case, seed):
    """The attentions from their definition in 64 bits, one sequence and KV head
    at a time.  What the other operators return is copied, not computed."""
    if case["op"] not in ("prompt", "tree"):
        return None
    s = prepare(case, seed)
    D, G, g = s["D"], s["G"], s["H"] // s["G"]
    out = torch.zeros_like(s["out"], dtype=torch.float64)
    for b in range(s["B"]):
        c, n = int(s["c"][b]), int(s["n"][b])
        if n == 0:
            continue
        if case["op"] == "prompt":
            a = int(s["cu"][b])
            q, k, v = s["q"][a:a + n].transpose(0, 1), s["k"][a:a + n].transpose(0, 1), s["v"][a:a + n].transpose(0, 1)
            marks = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        else:
            q, k, v = s["q"][b, :, :n], s["k"][b, :, :n], s["v"][b, :, :n]
            marks = s["seen"][b, :n, :n]
        for j in range(G):
            if "table" in s:
                page = s["table"][b, torch.arange(c, device="cuda") // PAGE].long()
                slot = torch.arange(c, device="cuda") % PAGE
                keys, vals = s["K"][0, page, j, slot], s["V"][0, page, j, slot]
            else:
                keys, vals = s["K"][0, b, j, :c], s["V"][0, b, j, :c]
            keys, vals = torch.cat([keys, k[j]]).double(), torch.cat([vals, v[j]]).double()
            see = torch.cat([torch.ones(n, c, dtype=torch.bool, device="cuda"), marks], 1)
            for i in range(j * g, j * g + g):
                score = (q[i].double() @ keys.T / D ** 0.5).masked_fill(~see, -math.inf)
                o = torch.softmax(score, -1) @ vals
                if case["op"] == "prompt":
                    out[a:a + n, i] = o
                else:
                    out[b, i, :n] = o
    return out
