"""Workloads of the window, paged-cache and cache-page operators.

Each case is one pass through one of them, as a training step, a prefill or a serving step makes it:

  window   sliding-window attention with sink tokens, forward alone (prefill)
  train    the same, forward and backward (a layer's attention in a training step)
  tree     attention of each sequence's newest tokens (one, a chain or a drafted tree) over a paged key/value cache
  branch   a speculative step on forked sequences: fork, append the drafted tokens, keep the accepted ones, free
  fill     prompts written into a paged cache, and the sequences freed again

With ``own`` false, ``run`` computes the operator from elementary torch operations in 32 bits; with ``own`` true it
calls the library.  ``exact`` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # a short chunk of a prompt against its context; lengths that divide nothing
        dict(name="window-chunk", kind="window", B=1, Hq=8, Hkv=2, Sq=500, Sk=1500, D=64, W=256, sinks=4, causal=1),
        # prefill of a long context
        dict(name="window-long", kind="window", B=1, Hq=32, Hkv=8, Sq=32768, Sk=32768, D=128, W=1024, sinks=4,
             causal=1),
        # a small training step, no sinks, a window that ends inside a tile
        dict(name="train-small", kind="train", B=2, Hq=16, Hkv=16, Sq=1000, Sk=1000, D=64, W=200, sinks=0, causal=1),
        # a long-context training step with grouped heads
        dict(name="train-long", kind="train", B=1, Hq=32, Hkv=8, Sq=16384, Sk=16384, D=128, W=1024, sinks=4,
             causal=1),
        # one request, one token: latency
        dict(name="decode-one", kind="tree", B=1, Hq=32, Hkv=8, D=128, n=1, L=2048, P=16, W=0, sinks=0, mask=False),
        # a serving batch, one token each, ragged contexts
        dict(name="decode-batch", kind="tree", B=64, Hq=32, Hkv=8, D=128, n=1, L=8192, P=64, W=0, sinks=0,
             mask=False),
        # drafted trees of up to 64 tokens
        dict(name="tree-64", kind="tree", B=8, Hq=32, Hkv=8, D=128, n=64, L=16384, P=32, W=0, sinks=0, mask=True),
        # streaming generation: long caches read through a window and the first tokens
        dict(name="decode-window", kind="tree", B=32, Hq=16, Hkv=16, D=64, n=1, L=32768, P=128, W=4096, sinks=4,
             mask=False),
        # a few candidates of one request
        dict(name="branch-small", kind="branch", Hkv=8, D=128, P=16, parents=1, fan=4, L=1000, n=8),
        # a batch of requests, each tried with several drafted continuations
        dict(name="branch-batch", kind="branch", Hkv=8, D=128, P=64, parents=32, fan=4, L=4096, n=33),
        # a short prompt enters the cache
        dict(name="fill-short", kind="fill", Hkv=8, D=64, P=32, rows=3, n=77),
        # long prompts enter the cache
        dict(name="fill-long", kind="fill", Hkv=8, D=128, P=64, rows=16, n=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["window", "train", "tree", "tree", "branch", "fill"])
    D = rng.choice([64, 128])
    Hkv, G = rng.choice([(1, 8), (2, 4), (8, 4), (8, 1), (4, 6), (16, 1), (2, 16)])
    if kind in ("window", "train"):
        Sq = _log(rng, 100, 12000 if kind == "window" else 6000)
        Sk = rng.choice([Sq, Sq, Sq + _log(rng, 1, 3000)])
        return dict(kind=kind, B=rng.choice([1, 1, 2]), Hq=Hkv * G, Hkv=Hkv, Sq=Sq, Sk=Sk, D=D,
                    W=_log(rng, 16, 2000), sinks=rng.choice([0, 1, 4, 130]), causal=rng.choice([1, 1, 2]))
    P = rng.choice([16, 32, 64, 128])
    if kind == "tree":
        mask = rng.random() < 0.5
        n = _log(rng, 2, 64) if mask else rng.choice([1, 1, 1, _log(rng, 2, 300)])
        B = _log(rng, 1, 48) if n <= 64 else _log(rng, 1, 4)
        W = rng.choice([0, 0, _log(rng, 100, 4000)])
        return dict(kind=kind, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, n=n, L=n + _log(rng, 1, 8000), P=P, W=W,
                    sinks=rng.choice([0, 4]) if W else 0, mask=mask)
    if kind == "branch":
        return dict(kind=kind, Hkv=Hkv, D=D, P=P, parents=_log(rng, 1, 32), fan=rng.choice([1, 2, 4]),
                    L=_log(rng, 10, 3500), n=_log(rng, 1, 64))
    return dict(kind=kind, Hkv=Hkv, D=D, P=P, rows=_log(rng, 1, 16), n=_log(rng, 1, 5000))


# ---------------------------------------------------------------------------- sizes a case implies
def _spread(case, salt, count, lo, hi):
    """``count`` whole numbers in [lo, hi] that depend on the case alone, hi itself the first."""
    r = np.random.RandomState((salt * 7919 + case["D"] * 31 + case["P"] * 17 + count * 131 + hi) % (1 << 31))
    x = r.randint(lo, hi + 1, size=count)
    x[0] = hi
    return x.astype(np.int64)


def _tree_sizes(case):
    n = _spread(case, 1, case["B"], max(1, case["n"] // 2), case["n"])
    lens = np.maximum(_spread(case, 2, case["B"], max(1, case["L"] // 2), case["L"]), n)
    return n, lens


def _parents(case, n):
    """Drafted trees: the parent of each token among its sequence's drafted ones (-1: the context)."""
    r = np.random.RandomState(int(n.sum()) + case["L"])
    return [np.array([r.randint(max(-1, u - 6), u) for u in range(m)]) for m in n]


def _visible(parents):
    """bool [m, m]: drafted tokens that token t sees: its ancestors and itself."""
    m = len(parents)
    vis = np.zeros((m, m), bool)
    for t in range(m):
        if parents[t] >= 0:
            vis[t] = vis[parents[t]]
        vis[t, t] = True
    return vis


def _window_counts(case):
    """Keys each query row sees."""
    i = np.arange(case["Sq"], dtype=np.int64)
    p = i + (case["Sk"] - case["Sq"] if case["causal"] == 1 else 0)
    hi = np.minimum(p, case["Sk"] - 1)
    lo = np.maximum(p - case["W"] + 1, 0)
    near = np.maximum(hi - lo + 1, 0)
    far = np.maximum(np.minimum(np.minimum(case["sinks"], lo), hi + 1), 0)
    return near + far


def work(case):
    if case["kind"] in ("window", "train"):
        pairs = float(_window_counts(case).sum()) * case["B"] * case["Hq"]
        q = case["B"] * case["Hq"] * case["Sq"]
        kv = case["B"] * case["Hkv"] * case["Sk"]
        fwd = 2 * 2 * case["D"] * (q + kv) + 4 * q
        if case["kind"] == "window":
            return {"bytes": fwd, "flops": 4 * case["D"] * pairs}
        return {"bytes": 2 * 2 * case["D"] * (q + kv) + 2 * case["D"] * (2 * q + 2 * kv) + 4 * q,
                "flops": 14 * case["D"] * pairs}
    if case["kind"] == "tree":
        n, lens = _tree_sizes(case)
        keys = pairs = 0.0
        for m, length in zip(n, lens):
            ctx = length - m
            seen = min(ctx, case["W"] + min(case["sinks"], max(0, ctx - case["W"]))) if case["W"] else ctx
            keys += seen + m
            pairs += m * (seen + (m + 1) / 2)
        t = float(n.sum())
        return {"bytes": 4 * case["D"] * case["Hkv"] * keys + 4 * case["D"] * case["Hq"] * t + 4 * case["Hq"] * t,
                "flops": 4 * case["D"] * case["Hq"] * pairs}
    row = 4 * case["Hkv"] * case["D"]  # one token's K and V, bf16
    if case["kind"] == "fill":
        n = _spread(case, 3, case["rows"], max(1, case["n"] // 2), case["n"])
        return {"bytes": float(2 * row * n.sum()), "flops": 0}
    lens, n, acc = _branch_sizes(case)
    moved = sum(int((a != np.arange(len(a))).sum()) for a in acc)
    part = np.repeat(lens % case["P"], case["fan"]).sum()
    return {"bytes": float(2 * row * (n.sum() + moved + part)), "flops": 0}


def _branch_sizes(case):
    lens = _spread(case, 4, case["parents"], max(1, case["L"] // 2), case["L"])
    n = _spread(case, 5, case["parents"] * case["fan"], max(1, case["n"] // 2), case["n"])
    r = np.random.RandomState(int(n.sum()) + case["L"])
    acc = [np.sort(r.choice(m, size=r.randint(1, m + 1), replace=False)) for m in n]
    return lens, n, acc


# ---------------------------------------------------------------------------- inputs
def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _cu(n):
    return np.concatenate([[0], np.cumsum(n)])


def _owners(n):
    """For packed tokens: the sequence of each and its place in it."""
    b = np.repeat(np.arange(len(n)), n)
    return b, np.arange(int(n.sum())) - _cu(n)[b]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    s = {"case": case}
    D, Hkv = case["D"], case["Hkv"]
    if case["kind"] in ("window", "train"):
        s["q"] = normal(case["B"], case["Hq"], case["Sq"], D)
        s["k"] = normal(case["B"], Hkv, case["Sk"], D)
        s["v"] = normal(case["B"], Hkv, case["Sk"], D)
        if case["kind"] == "train":
            s["dout"] = normal(case["B"], case["Hq"], case["Sq"], D)
        return s
    P = case["P"]
    r = np.random.RandomState(int(seed) % (1 << 31))
    if case["kind"] == "tree":
        n, lens = _tree_sizes(case)
        used = -(-lens // P)
        n_pages = int(used.sum()) + 7
    elif case["kind"] == "branch":
        par, n, acc = _branch_sizes(case)
        kids = len(n)
        used = np.concatenate([-(-par // P), np.zeros(kids, np.int64)])
        lens = np.concatenate([par, np.zeros(kids, np.int64)])
        per_kid = -(-case["n"] // P) + 2
        n_pages = int(used.sum()) + kids * per_kid
        n = np.concatenate([np.zeros(len(par), np.int64), n])
    else:
        n = _spread(case, 3, case["rows"], max(1, case["n"] // 2), case["n"])
        lens = np.zeros(case["rows"], np.int64)
        used = lens
        n_pages = int((-(-n // P)).sum()) + 5
    width = int(max((-(-(lens + (n if case["kind"] == "fill" else 0)) // P)).max(), 1))
    if case["kind"] == "branch":
        width += -(-case["n"] // P) + 1
    table = np.full((len(lens), width), -1, np.int64)
    order = r.permutation(n_pages)
    ref = np.zeros(n_pages, np.int64)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        ref[order[at:at + u]] = 1
        at += u
    s["k_pages"] = normal(n_pages, Hkv, P, D)
    s["v_pages"] = normal(n_pages, Hkv, P, D)
    s["page_table"] = _i32(table)
    s["seq_lens"] = _i32(lens)
    s["cu_tokens"] = _i32(_cu(n))
    owner, place = _owners(n)
    s["owner"] = torch.as_tensor(owner, device="cuda")
    s["place"] = torch.as_tensor(place, device="cuda")
    s["n_max"] = int(n.max())
    if case["kind"] == "tree":
        s["q"] = normal(int(n.sum()), case["Hq"], D)
        s["tree_mask"] = None
        if case["mask"]:
            words = -(-case["n"] // 32)
            bits = np.zeros((int(n.sum()), words * 32), np.uint64)
            for c, pa in zip(_cu(n), _parents(case, n)):
                bits[c:c + len(pa), :len(pa)] = _visible(pa)
            packed = (bits.reshape(-1, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
            s["tree_mask"] = torch.as_tensor(packed.astype(np.uint32).view(np.int32), device="cuda")
        return s
    s["ref_counts"] = _i32(ref)
    s["k_new"] = normal(int(n.sum()), Hkv, D)
    s["v_new"] = normal(int(n.sum()), Hkv, D)
    if case["kind"] == "branch":
        kids = np.arange(len(par), len(lens))
        s["parents"] = _i32(np.repeat(np.arange(len(par)), case["fan"]))
        s["children"] = _i32(kids)
        s["accepted"] = _i32(np.concatenate(acc))
        counts = np.concatenate([np.zeros(len(par), np.int64), [len(a) for a in acc]])
        s["cu_accepted"] = _i32(_cu(counts))
        b, i = _owners(counts)
        s["acc_owner"] = torch.as_tensor(b, device="cuda")
        s["acc_place"] = torch.as_tensor(i, device="cuda")
    else:
        s["rows"] = _i32(np.arange(case["rows"]))
    return s


# ---------------------------------------------------------------------------- plain forms
def _bands(s):
    """Queries in blocks of C rows, the keys of each block's window (and the sinks) gathered beside it."""
    c = s["case"]
    B, Hq, Hkv, Sq, Sk, D = (c[x] for x in ("B", "Hq", "Hkv", "Sq", "Sk", "D"))
    C, W = 512, min(c["W"], c["Sk"] + c["Sq"])
    nb = -(-Sq // C)
    dev = s["q"].device
    diag = Sk - Sq if c["causal"] == 1 else 0
    first = torch.arange(nb, device=dev)[:, None] * C + diag
    near = first + torch.arange(W + C - 1, device=dev)[None] - (W - 1)
    sink = torch.arange(min(c["sinks"], Sk), device=dev)[None].expand(nb, -1)
    keys = torch.cat([near, sink], 1)
    p = (first + torch.arange(C, device=dev)[None])[:, :, None]
    inside = (keys >= 0) & (keys < Sk)
    is_sink = torch.arange(keys.shape[1], device=dev) >= near.shape[1]
    dist = p - keys[:, None, :]
    seen = inside[:, None, :] & (dist >= 0) & ((dist < W) != is_sink)
    keys = keys.clamp(0, max(Sk - 1, 0))

    def rows(x):
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, nb * C - Sq))
        return x.view(B, Hkv, Hq // Hkv, nb, C, D).transpose(2, 3).reshape(B, Hkv, nb, -1, D)

    def back(x):
        x = x.view(B, Hkv, nb, Hq // Hkv, C, -1).transpose(2, 3).reshape(B, Hq, nb * C, -1)
        return x[:, :, :Sq]

    return rows, back, keys, seen.repeat(1, Hq // Hkv, 1), C


def _plain_window(s, backward):
    rows, back, keys, seen, _ = _bands(s)
    q, k, v = rows(s["q"]), s["k"].float()[:, :, keys], s["v"].float()[:, :, keys]
    scale = s["case"]["D"] ** -0.5
    logits = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)))
    total = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    o = torch.matmul(p, v)
    lse = back(top + torch.log(total))[..., 0].contiguous()
    out = {"o": back(o).to(torch.bfloat16), "lse": lse}
    if backward:
        do = rows(s["dout"])
        at = keys.reshape(-1)

        def gather(x):
            return torch.zeros_like(s["k"], dtype=torch.float32).index_add_(2, at, x.flatten(2, 3))

        out["dv"] = gather(torch.matmul(p.transpose(-1, -2), do)).to(torch.bfloat16)
        ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        out["dq"] = back(torch.matmul(ds, k)).to(torch.bfloat16)
        out["dk"] = gather(torch.matmul(ds.transpose(-1, -2), q)).to(torch.bfloat16)
    return out


def _plain_tree(s):
    c = s["case"]
    B, Hq, Hkv, D, P = (c[x] for x in ("B", "Hq", "Hkv", "D", "P"))
    dev, G, m = s["q"].device, Hq // Hkv, s["n_max"]
    table, lens = s["page_table"].long().clamp(min=0), s["seq_lens"].long()
    n = (s["cu_tokens"][1:] - s["cu_tokens"][:-1]).long()
    ctx = lens - n

    def cache(x):  # [B, Hkv, L, D]
        return x[table].float().transpose(1, 2).reshape(B, Hkv, -1, D)

    q = torch.zeros((B, m, Hq, D), device=dev)
    q[s["owner"], s["place"]] = s["q"].float()
    q = q.view(B, m, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, m * G, D)
    k = cache(s["k_pages"])
    j = torch.arange(k.shape[2], device=dev)[None, None]
    u = j - ctx[:, None, None]  # the drafted token that a key belongs to, below 0 for the context
    t = torch.arange(m, device=dev)[None, :, None]
    if s["tree_mask"] is not None:
        words = torch.zeros((B, m, s["tree_mask"].shape[1]), dtype=torch.long, device=dev)
        words[s["owner"], s["place"]] = s["tree_mask"].long()
        bits = ((words[..., None] >> torch.arange(32, device=dev)) & 1).flatten(2)
        bits = bits * (torch.arange(bits.shape[2], device=dev) < n[:, None, None])
        at = u.clamp(0, bits.shape[2] - 1).expand(B, m, -1)
        seen = (u < 0) | ((u < n[:, None, None]) & (torch.gather(bits, 2, at) > 0))
        depth = bits.sum(-1, keepdim=True) - 1
    else:
        seen = u <= t
        depth = t
    if c["W"]:
        near = (ctx[:, None, None] + depth - j < c["W"]) | (j < c["sinks"])
        seen = seen & (near if s["tree_mask"] is None else (near | (u >= 0)))
    seen = (seen & (j < lens[:, None, None])).repeat_interleave(G, 1)[:, None]
    logits = torch.matmul(q, k.transpose(-1, -2)).mul_(D ** -0.5).masked_fill_(~seen, -math.inf)
    del k
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, cache(s["v_pages"])) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total)).view(B, Hkv, m, G).transpose(1, 2).reshape(B, m, Hq)
    o = o.view(B, Hkv, m, G, D).transpose(1, 2).reshape(B, m, Hq, D)
    return {"o": o[s["owner"], s["place"]].to(torch.bfloat16), "lse": lse[s["owner"], s["place"]]}


def _count(s, pages, keep, by):
    """Reference counts of the kept pages changed by ``by``."""
    ref = s["ref_counts"]
    at = torch.where(keep, pages.long(), ref.numel()).flatten()
    more = torch.zeros(ref.numel() + 1, dtype=torch.int32, device=ref.device)
    ref.add_(more.index_add_(0, at, torch.full_like(at, by, dtype=torch.int32))[:-1])


def _take(s, want):
    """The lowest free pages, one for each true place of ``want`` in order."""
    free = torch.argsort((s["ref_counts"] > 0).to(torch.int32), stable=True).to(torch.int32)
    nth = torch.cumsum(want.flatten().long(), 0).sub(1).clamp(min=0).view(want.shape)
    got = torch.where(want, free[nth], -1)
    _count(s, got, want, 1)
    return got


def _fork(s):
    P, table = s["case"]["P"], s["page_table"]
    dad, kid = s["parents"].long(), s["children"].long()
    lens = s["seq_lens"][dad]
    at = torch.arange(table.shape[1], device=table.device)[None]
    full, part = (lens // P)[:, None], (lens % P)[:, None]
    share, last = at < full, (at == full) & (part > 0)
    old = table[dad]
    _count(s, old, share, 1)
    new = _take(s, last)
    table[kid] = torch.where(share, old, new)
    src = torch.where(last, old, 0).sum(1).long()
    dst = torch.where((part > 0)[:, 0], torch.where(last, new, 0).sum(1).long(), src)
    inside = (torch.arange(P, device=table.device) < part)[:, None, :, None]
    for x in (s["k_pages"], s["v_pages"]):
        x[dst] = torch.where(inside, x[src], x[dst])
    s["seq_lens"][kid] = lens


def _append(s):
    P, table, before = s["case"]["P"], s["page_table"], s["seq_lens"].clone()
    s["seq_lens"].add_(s["cu_tokens"][1:] - s["cu_tokens"][:-1])
    at = torch.arange(table.shape[1], device=table.device)[None]
    want = (at >= ((before + P - 1) // P)[:, None]) & (at < ((s["seq_lens"] + P - 1) // P)[:, None])
    table.copy_(torch.where(want, _take(s, want), table))
    pos = before[s["owner"]].long() + s["place"]
    page = table[s["owner"], pos // P].long()
    s["k_pages"][page, :, pos % P] = s["k_new"]
    s["v_pages"][page, :, pos % P] = s["v_new"]


def _drop(s, rows, keep):
    """Pages of ``rows`` past the first ``keep`` tokens given back."""
    P, table = s["case"]["P"], s["page_table"]
    at = torch.arange(table.shape[1], device=table.device)[None]
    had = ((s["seq_lens"][rows] + P - 1) // P)[:, None]
    gone = (at >= ((keep + P - 1) // P)[:, None]) & (at < had)
    _count(s, table[rows], gone, -1)
    table[rows] = torch.where(gone, -1, table[rows])
    s["seq_lens"][rows] = keep


def _compact(s):
    P, table = s["case"]["P"], s["page_table"]
    ctx = (s["seq_lens"] - (s["cu_tokens"][1:] - s["cu_tokens"][:-1])).long()
    b = s["acc_owner"]
    src, dst = ctx[b] + s["accepted"].long(), ctx[b] + s["acc_place"]
    sp, dp = table[b, src // P].long(), table[b, dst // P].long()
    for x in (s["k_pages"], s["v_pages"]):
        x[dp, :, dst % P] = x[sp, :, src % P]
    kept = ctx.to(torch.int32) + (s["cu_accepted"][1:] - s["cu_accepted"][:-1])
    _drop(s, torch.arange(table.shape[0], device=table.device), kept)


def _free(s, rows):
    _drop(s, rows.long(), torch.zeros_like(rows))


# ---------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        from attention_forward_06_gb300 import ops
    if c["kind"] in ("window", "train"):
        if not own:
            return _plain_window(s, c["kind"] == "train")
        o, lse = ops.attn_fwd_window(s["q"], s["k"], s["v"], c["W"], sinks=c["sinks"], causal=c["causal"])
        out = {"o": o, "lse": lse}
        if c["kind"] == "train":
            out["dq"], out["dk"], out["dv"] = ops.attn_bwd_window(
                s["q"], s["k"], s["v"], o, lse, s["dout"], c["W"], sinks=c["sinks"], causal=c["causal"])
        return out
    if c["kind"] == "tree":
        if not own:
            return _plain_tree(s)
        if "workspace" not in s:
            s["workspace"] = torch.empty(ops.tree_workspace_size(c["D"]), dtype=torch.uint8, device="cuda")
        o, lse = ops.attn_fwd_tree(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"],
                                   s["cu_tokens"], tree_mask=s["tree_mask"], window=c["W"], sinks=c["sinks"],
                                   workspace=s["workspace"])
        return {"o": o, "lse": lse}
    pool = (s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"], s["ref_counts"])
    if c["kind"] == "branch":
        if own:
            ops.kv_fork(*pool, s["parents"], s["children"])
            ops.kv_append(s["k_new"], s["v_new"], *pool, s["cu_tokens"])
            ops.kv_compact(*pool, s["cu_tokens"], s["accepted"], s["cu_accepted"])
        else:
            _fork(s)
            _append(s)
            _compact(s)
        table, lens, rows = s["page_table"].clone(), s["seq_lens"].clone(), s["children"]
    else:
        if own:
            ops.kv_append(s["k_new"], s["v_new"], *pool, s["cu_tokens"])
        else:
            _append(s)
        table, lens, rows = s["page_table"].clone(), s["seq_lens"].clone(), s["rows"]
    if own:
        ops.kv_free(s["page_table"], s["seq_lens"], s["ref_counts"], rows, s["case"]["P"])
    else:
        _free(s, rows)
    return {"table": table, "lens": lens, "k_pages": s["k_pages"], "v_pages": s["v_pages"],
            "page_table": s["page_table"], "seq_lens": s["seq_lens"], "ref_counts": s["ref_counts"]}


# ---------------------------------------------------------------------------- the definition, in 64 bits
def _softmax64(x):
    top = x.amax(-1, keepdim=True) if x.shape[-1] else x.new_full(x.shape[:-1] + (1,), -math.inf)
    top0 = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(x - top0)
    z = e.sum(-1, keepdim=True)
    return e / torch.where(z > 0, z, torch.ones_like(z)), (top0 + torch.log(z))[..., 0]


def _exact_window(s):
    c = s["case"]
    B, Hq, Hkv, Sq, Sk, D, W = (c[x] for x in ("B", "Hq", "Hkv", "Sq", "Sk", "D", "W"))
    G, scale, diag = Hq // Hkv, D ** -0.5, Sk - Sq if c["causal"] == 1 else 0
    dev = s["q"].device
    o = torch.zeros((B, Hq, Sq, D), dtype=torch.float64, device=dev)
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64, device=dev)
    train = c["kind"] == "train"
    if train:
        dq, dk, dv = (torch.zeros(s[x].shape, dtype=torch.float64, device=dev) for x in "qkv")
    for b in range(B):
        for h in range(Hkv):
            heads = slice(h * G, h * G + G)
            kk, vv = s["k"][b, h].double(), s["v"][b, h].double()
            for i0 in range(0, Sq, 1024):
                i1 = min(i0 + 1024, Sq)
                lo, hi = max(0, i0 + diag - W + 1), max(0, min(Sk, i1 + diag))
                lo = min(lo, hi)
                j = torch.cat([torch.arange(0, min(c["sinks"], lo), device=dev), torch.arange(lo, hi, device=dev)])
                if j.numel() == 0:
                    continue
                gap = (torch.arange(i0, i1, device=dev) + diag)[:, None] - j[None]
                ok = (gap >= 0) & ((gap < W) | (j < c["sinks"])[None])
                qq = s["q"][b, heads, i0:i1].double()
                x = (qq @ kk[j].T * scale).masked_fill(~ok, -math.inf)
                p, z = _softmax64(x)
                oo = p @ vv[j]
                o[b, heads, i0:i1], lse[b, heads, i0:i1] = oo, z
                if train:
                    do = s["dout"][b, heads, i0:i1].double()
                    dv[b, h].index_add_(0, j, torch.einsum("gij,gid->jd", p, do))
                    d = p * (do @ vv[j].T - (do * oo).sum(-1, keepdim=True)) * scale
                    dq[b, heads, i0:i1] = d @ kk[j]
                    dk[b, h].index_add_(0, j, torch.einsum("gij,gid->jd", d, qq))
    out = {"o": o, "lse": lse}
    return dict(out, dq=dq, dk=dk, dv=dv) if train else out


def _exact_tree(s):
    c = s["case"]
    Hq, Hkv, D, P = (c[x] for x in ("Hq", "Hkv", "D", "P"))
    n, lens = _tree_sizes(c)
    cu, G, dev = _cu(n), Hq // Hkv, s["q"].device
    trees = [_visible(p) for p in _parents(c, n)] if c["mask"] else [np.tril(np.ones((m, m), bool)) for m in n]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=dev)
    for b, (m, length) in enumerate(zip(n.tolist(), lens.tolist())):
        ctx = length - m
        pages = s["page_table"][b, :-(-length // P)].long()
        ok = np.ones((m, length), bool)
        ok[:, ctx:] = trees[b]
        if c["W"]:
            pos = ctx + trees[b].sum(1) - 1
            near = (pos[:, None] - np.arange(length)[None] < c["W"]) | (np.arange(length) < c["sinks"])[None]
            ok &= near if not c["mask"] else (near | (np.arange(length) >= ctx)[None])
        ok = torch.as_tensor(ok, device=dev)
        for h in range(Hkv):
            kk = s["k_pages"][pages, h].double().reshape(-1, D)[:length]
            vv = s["v_pages"][pages, h].double().reshape(-1, D)[:length]
            qq = s["q"][cu[b]:cu[b + 1], h * G:h * G + G].double()
            p, z = _softmax64((qq @ kk.T * D ** -0.5).masked_fill(~ok[:, None], -math.inf))
            o[cu[b]:cu[b + 1], h * G:h * G + G], lse[cu[b]:cu[b + 1], h * G:h * G + G] = p @ vv, z
    return {"o": o, "lse": lse}


def exact(case, seed):
    if case["kind"] in ("window", "train"):
        return _exact_window(prepare(case, seed))
    if case["kind"] == "tree":
        return _exact_tree(prepare(case, seed))
    return None  # rows are moved, nothing is computed
