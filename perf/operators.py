"""Operators around the decode step's paged latent cache, as they are measured.

  prefix    csa_prefix_attn: one token of each request of a batch whose requests share their first rows
            (a prompt sampled many times, beams), the shared rows attended once for the whole batch
  window    csa_window_attn: causal attention over a sliding window of the raw cache and the first tokens
            of the sequence (sinks), for prompt chunks of any length and for single tokens
  fork      csa_pages_free, csa_pages_fork: the page tables of a batch taken back and forked again
            from their parents, with a copy of each parent's last, partly filled page
  compact   csa_pages_compact: the pages in use moved to the front of the pools

Latent rows are bf16 [512] with K = V = the row, 64-token pages unless a case says otherwise.
`own` false: plain torch in 32 bits.  `own` true: the package's entry points.
"""
import math

import torch

own = False

D = 512
SCALE = 1.0 / math.sqrt(D)
POOLS = (64 * 512, 16 * 512, 16 * 128)  # bf16 values of a page: raw rows, compressed rows (4:1), index keys


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # two samples of a short prompt, 16 heads (the rest of the heads on other devices): latency
        {"name": "prefix-2x16-500", "op": "prefix", "B": 2, "H": 16, "shared": 500, "own": 40, "rpp": 64},
        # eight samples of an 8K prompt, every head on the device
        {"name": "prefix-8x128-8K", "op": "prefix", "B": 8, "H": 128, "shared": 8192, "own": 512, "rpp": 64},
        # 32 requests under a 64K document, 16 heads
        {"name": "prefix-32x16-64K", "op": "prefix", "B": 32, "H": 16, "shared": 65536, "own": 2048, "rpp": 64},
        # 32 requests under a 32K document, every head: the largest
        {"name": "prefix-32x128-32K", "op": "prefix", "B": 32, "H": 128, "shared": 32768, "own": 300, "rpp": 64},
        # one token of one request: latency
        {"name": "window-decode-1x128", "op": "window", "B": 1, "H": 128, "q": 1, "ctx": 4096, "window": 128,
         "sink": 4, "rpp": 64},
        # one token of each of 64 ragged requests, pages behind the window already given back
        {"name": "window-decode-64x16", "op": "window", "B": 64, "H": 16, "q": 1, "ctx": 131072, "window": 128,
         "sink": 16, "rpp": 64},
        # a prompt of 8K tokens
        {"name": "window-prefill-8K", "op": "window", "B": 1, "H": 128, "q": 8192, "ctx": 0, "window": 128,
         "sink": 4, "rpp": 64},
        # ragged chunks of seven prompts, a wide window, pages that are no multiple of 16 rows
        {"name": "window-chunks-7x24", "op": "window", "B": 7, "H": 24, "q": 700, "ctx": 5000, "window": 512,
         "sink": 5, "rpp": 40},
        # a 4K prompt forked into four samples: latency
        {"name": "fork-1-to-4-4K", "op": "fork", "parents": 1, "children": 4, "tokens": 4090, "pages": 256},
        # two 512K contexts, eight branches of each
        {"name": "fork-2-to-16-512K", "op": "fork", "parents": 2, "children": 16, "tokens": 524000,
         "pages": 20000},
        # a small cache: latency
        {"name": "compact-256", "op": "compact", "B": 4, "pages": 256, "used": 0.25},
        # a cache of 16K pages, a little over half of it in use
        {"name": "compact-16K", "op": "compact", "B": 32, "pages": 16384, "used": 0.6},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("prefix", "prefix", "window", "window", "fork", "compact"))
    rpp = rng.choice((64, 64, 64, 16, 48, 128, 40, 17, 1))
    if op == "prefix":
        B, H = _log(rng, 1, 32), rng.choice((rng.randint(1, 128), 16, 64, 128))
        shared = _log(rng, 1, min(131072, 4096 * 32768 // (B * H)))
        return {"op": op, "B": B, "H": H, "shared": shared, "own": _log(rng, 1, 2048), "rpp": rpp}
    if op == "window":
        H, window, sink = rng.choice((rng.randint(1, 128), 16, 64, 128)), _log(rng, 1, 1024), rng.randint(0, 64)
        B = _log(rng, 1, 64)
        most = min(8192 * 128 * 132 // (H * (window + sink)), 2000000 // (window + sink), 8192)
        q = 1 if rng.random() < 0.3 else _log(rng, 1, max(1, most // B))
        return {"op": op, "B": B, "H": H, "q": q, "ctx": rng.choice((0, _log(rng, 1, 131072))), "window": window,
                "sink": sink, "rpp": rpp}
    if op == "fork":
        parents, children = _log(rng, 1, 16), _log(rng, 1, 64)
        tokens = _log(rng, 1, 524000)
        tokens = max(1, min(tokens, 64 * 16000 // parents))
        return {"op": op, "parents": parents, "children": max(parents, children), "tokens": tokens,
                "pages": parents * (tokens // 64 + 1) + max(parents, children) + _log(rng, 1, 2000)}
    return {"op": op, "B": _log(rng, 1, 32), "pages": _log(rng, 40, 16384), "used": round(rng.uniform(0.05, 0.95), 3)}


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _lengths(g, n, most, least):
    """n lengths of [least, most], the longest among them."""
    v = torch.randint(least, most + 1, (n,), generator=g, device="cuda", dtype=torch.int64)
    v[n // 2] = most
    return v


def _chunks(c):
    """New tokens of each sequence: ragged, the same for every seed (they are the outputs' shape)."""
    v = [1 + int((0.381966 * (i + 1)) % 1.0 * c["q"]) for i in range(c["B"])]
    v[c["B"] // 2] = c["q"]
    return v


def prepare(case, seed):
    return {"prefix": _prepare_prefix, "window": _prepare_window, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, seed)


def _prepare_prefix(c, seed):
    g = _gen(seed)
    B, H, shared, rpp = c["B"], c["H"], c["shared"], c["rpp"]
    n_rows = shared + _lengths(g, B, c["own"], 0)
    full = shared // rpp                                  # whole pages that every request's table names
    width = (shared + c["own"] + rpp - 1) // rpp
    mine = width - full
    n_pages = full + B * mine + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.empty(B, width, dtype=torch.int32, device="cuda")
    table[:, :full] = perm[:full]
    table[:, full:] = perm[full: full + B * mine].view(B, mine)
    pool = _randn(g, n_pages * rpp, D)
    part = shared - full * rpp                            # the page that ends the prefix, copied by the fork
    if part:
        v = pool.view(n_pages, rpp, D)
        v[table[:, full].long(), :part] = v[table[0, full].long(), :part].unsqueeze(0)
    q = _randn(g, B, H, D)
    return {"case": c, "q": q, "pool": pool, "table": table, "n_rows": n_rows, "n_pages": n_pages,
            "max_rows": shared + c["own"], "out": torch.zeros_like(q),
            "lse": torch.zeros(B, H, dtype=torch.float32, device="cuda")}


def _prepare_window(c, seed):
    g = _gen(seed)
    B, H, rpp, W, S = c["B"], c["H"], c["rpp"], c["window"], c["sink"]
    q_len = torch.tensor(_chunks(c), dtype=torch.int64, device="cuda")
    before = _lengths(g, B, c["ctx"], min(c["ctx"], 1)) if c["ctx"] else torch.zeros_like(q_len)
    n_tokens = q_len + before
    offsets = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(q_len, 0)
    total = sum(_chunks(c))
    width = (c["q"] + c["ctx"] + rpp - 1) // rpp
    page = torch.arange(width, device="cuda").view(1, width)
    first = (before + 1 - W).clamp(min=0) // rpp          # the first page that a window still reaches
    live = (page * rpp < n_tokens.view(B, 1)) & ((page >= first.view(B, 1)) | (page * rpp < S))
    rank = torch.cumsum(live.view(-1), 0).view(B, width) - 1
    used = int(live.sum())
    perm = torch.randperm(used + 2, generator=g, device="cuda").to(torch.int32)
    table = torch.where(live, perm[rank.clamp(min=0)], torch.full_like(perm[:1], -1)).contiguous()
    pool = _randn(g, (used + 2) * rpp, D)
    q = _randn(g, total, H, D)
    return {"case": c, "q": q, "pool": pool, "table": table, "n_tokens": n_tokens, "offsets": offsets,
            "n_pages": used + 2, "max_q": c["q"], "out": torch.zeros_like(q),
            "lse": torch.zeros(total, H, dtype=torch.float32, device="cuda")}


def _pools(g, n_pages):
    return [torch.randint(-32768, 32768, (n_pages, w), generator=g, device="cuda", dtype=torch.int16) for w in POOLS]


def _prepare_fork(c, seed):
    g = _gen(seed)
    P, F, n_pages = c["parents"], c["children"], c["pages"]
    width = c["tokens"] // 64 + 1
    n_tokens = torch.zeros(P + F, dtype=torch.int64, device="cuda")
    n_tokens[:P] = _lengths(g, P, c["tokens"], (c["tokens"] + 1) // 2)
    pages = (n_tokens[:P] + 63) // 64
    live = torch.arange(width, device="cuda").view(1, width) < pages.view(P, 1)
    rank = torch.cumsum(live.view(-1), 0).view(P, width) - 1
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((P + F, width), -1, dtype=torch.int32, device="cuda")
    table[:P] = torch.where(live, perm[rank.clamp(min=0)], table[:P])
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs.scatter_add_(0, table[:P].reshape(-1).clamp(min=0).long(), live.reshape(-1).int())
    dst = torch.arange(P, P + F, dtype=torch.int32, device="cuda")
    src = torch.randint(0, P, (F,), generator=g, device="cuda", dtype=torch.int32)
    return {"case": c, "pools": _pools(g, n_pages), "table": table, "refs": refs, "n_tokens": n_tokens, "src": src,
            "dst": dst}


def _prepare_compact(c, seed):
    g = _gen(seed)
    B, n_pages = c["B"], c["pages"]
    used = max(1, int(n_pages * c["used"]))
    width = (used + B - 1) // B + 1
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    k = torch.arange(used, device="cuda")
    table[k % B, k // B] = perm[:used]
    table[:, width - 1] = table[:, 0].clamp(min=-1).roll(1)  # a page that another request's table names too
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    flat = table.reshape(-1)
    refs.scatter_add_(0, flat.clamp(min=0).long(), (flat >= 0).int())
    return {"case": c, "pools": _pools(g, n_pages), "table": table, "refs": refs,
            "table_out": torch.empty_like(table), "refs_out": torch.empty_like(refs),
            "n_used": torch.zeros(1, dtype=torch.int64, device="cuda")}


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _softmax_parts(parts):
    """Rows of several blocks of logits under one softmax: the weights of each block, and the log of the sum."""
    m = torch.stack([p.amax(-1) for p in parts]).amax(0)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    e = [torch.exp(p - m.unsqueeze(-1)) for p in parts]
    total = sum(x.sum(-1) for x in e)
    return e, total, m + torch.log(total)


def _plain_prefix(s):
    c, table = s["case"], s["table"].long()
    B, H, P, rpp = c["B"], c["H"], c["shared"], c["rpp"]
    j = torch.arange(P, device="cuda")
    head = s["pool"][table[0, j // rpp] * rpp + j % rpp].float()
    j = torch.arange(P, s["max_rows"], device="cuda")
    mine = s["pool"][table[:, j // rpp] * rpp + j % rpp].float()          # [B, own, 512]
    q = s["q"].float() * SCALE
    a = (q.view(B * H, D) @ head.t()).view(B, H, P)
    b = torch.bmm(q, mine.transpose(1, 2))
    b = b.masked_fill((j.view(1, -1) >= s["n_rows"].view(B, 1)).unsqueeze(1), float("-inf"))
    (ea, eb), total, lse = _softmax_parts((a, b))
    o = (ea.view(B * H, P) @ head).view(B, H, D) + torch.bmm(eb, mine)
    return {"out": (o / total.unsqueeze(-1)).to(torch.bfloat16), "lse": lse}


def _plain_window(s):
    c, table = s["case"], s["table"].long()
    B, H, W, S, rpp = c["B"], c["H"], c["window"], c["sink"], c["rpp"]
    T = s["q"].shape[0]
    i = torch.arange(T, device="cuda")
    b = torch.bucketize(i, s["offsets"][1:], right=True)
    pos = s["n_tokens"][b] - (s["offsets"][b + 1] - i)
    win = pos.view(T, 1) - (W - 1) + torch.arange(W, device="cuda")
    first = torch.arange(S, device="cuda").expand(T, S)
    key = torch.cat([first, win], 1)
    seen = torch.cat([first < win[:, :1].clamp(min=0), win >= 0], 1)
    key = torch.where(seen, key, pos.view(T, 1))
    rows = table[b.view(T, 1), key // rpp] * rpp + key % rpp
    kv = s["pool"][rows].float()                                          # [T, S + W, 512]
    a = torch.bmm(s["q"].float() * SCALE, kv.transpose(1, 2))
    a = a.masked_fill(~seen.unsqueeze(1), float("-inf"))
    (e,), total, lse = _softmax_parts((a,))
    o = torch.bmm(e, kv) / total.unsqueeze(-1)
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _plain_fork(s):
    table, refs, src, dst = s["table"], s["refs"], s["src"].long(), s["dst"].long()
    n_pages, width = refs.shape[0], table.shape[1]
    old = table[dst].reshape(-1)
    refs.scatter_add_(0, old.clamp(min=0).long(), -(old >= 0).int())
    n = s["n_tokens"][src]
    full, part = n // 64, n % 64 > 0
    rows, j = table[src], torch.arange(width, device="cuda")
    share = j < full.view(-1, 1)
    ids = torch.arange(n_pages, device="cuda")
    free = torch.sort(torch.where(refs == 0, ids, ids + n_pages)).values
    new = free[(torch.cumsum(part, 0) - 1).clamp(min=0)]
    last = rows.gather(1, full.clamp(max=width - 1).view(-1, 1)).view(-1).clamp(min=0).long()
    to = torch.where(part, new, last)
    refs.scatter_add_(0, rows.reshape(-1).clamp(min=0).long(), share.reshape(-1).int())
    refs.scatter_add_(0, to, part.int())
    fresh = (j == full.view(-1, 1)) & part.view(-1, 1)
    table[dst] = torch.where(share, rows, torch.where(fresh, to.view(-1, 1).int(), torch.full_like(rows, -1)))
    s["n_tokens"][dst] = n
    for p in s["pools"]:
        p[to] = p[last]
    return {"table": table, "refs": refs, "n_tokens": s["n_tokens"], "pools": s["pools"]}


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    ids = torch.arange(refs.shape[0], device="cuda")
    used = refs > 0
    n = used.sum()
    src, dst = (used & (ids >= n)).nonzero().view(-1), (~used & (ids < n)).nonzero().view(-1)
    to = ids.clone()
    to[src] = dst
    for p in s["pools"]:
        p[dst] = p[src]
    s["table_out"].copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    s["refs_out"].copy_(refs)
    s["refs_out"][dst] = refs[src]
    s["refs_out"][src] = 0
    s["n_used"].copy_(n)
    return {"table": s["table_out"], "refs": s["refs_out"], "n_used": s["n_used"], "pools": s["pools"]}


_PLAIN = {"prefix": _plain_prefix, "window": _plain_window, "fork": _plain_fork, "compact": _plain_compact}


def _scratch(s, nbytes):
    """The program's workspace: allocated once, for the calls that follow."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(16, nbytes), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own_prefix(s):
    import deepseek_v4_hybrid_c4_gb300 as m
    c = s["case"]
    B, H, P = c["B"], c["H"], c["shared"]
    if "kv" not in s:
        s["kv"] = m.paged(s["pool"], c["rpp"], 1024, s["table"], n_pages=s["n_pages"])
        s["bytes"] = m.csa_prefix_attn_workspace_size(B, H, P, s["max_rows"])
    m.csa_prefix_attn(s["q"], B, H, SCALE, s["kv"], s["table"].shape[1], P, s["n_rows"], s["max_rows"], s["out"],
                      s["lse"], _scratch(s, s["bytes"]), s["bytes"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_window(s):
    import deepseek_v4_hybrid_c4_gb300 as m
    c = s["case"]
    B, H, W, S, T = c["B"], c["H"], c["window"], c["sink"], s["q"].shape[0]
    if "kv" not in s:
        s["kv"] = m.paged(s["pool"], c["rpp"], 1024, s["table"], n_pages=s["n_pages"])
        s["bytes"] = m.csa_window_attn_workspace_size(B, H, T, s["max_q"], W, S)
    m.csa_window_attn(s["q"], H, SCALE, s["kv"], s["table"].shape[1], B, s["offsets"], s["n_tokens"], T, s["max_q"],
                      W, S, s["out"], s["lse"], _scratch(s, s["bytes"]), s["bytes"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_fork(s):
    import deepseek_v4_hybrid_c4_gb300 as m
    table, refs, F = s["table"], s["refs"], s["src"].shape[0]
    B, width = table.shape
    if "desc" not in s:
        s["desc"] = m.page_pools(s["pools"], refs.shape[0])
        s["bytes"] = m.csa_pages_workspace_size(refs.shape[0])
    m.csa_pages_free(refs, refs.shape[0], table, width, B, s["dst"], F)
    m.csa_pages_fork(s["desc"], refs, table, width, B, s["src"], s["dst"], F, s["n_tokens"], 64,
                     _scratch(s, s["bytes"]), s["bytes"])
    return {"table": table, "refs": refs, "n_tokens": s["n_tokens"], "pools": s["pools"]}


def _own_compact(s):
    import deepseek_v4_hybrid_c4_gb300 as m
    table, refs = s["table"], s["refs"]
    B, width = table.shape
    if "desc" not in s:
        s["desc"] = m.page_pools(s["pools"], refs.shape[0])
        s["bytes"] = m.csa_pages_workspace_size(refs.shape[0])
    m.csa_pages_compact(s["desc"], refs, s["refs_out"], table, s["table_out"], width, B, s["n_used"],
                        _scratch(s, s["bytes"]), s["bytes"])
    return {"table": s["table_out"], "refs": s["refs_out"], "n_used": s["n_used"], "pools": s["pools"]}


_OWN = {"prefix": _own_prefix, "window": _own_window, "fork": _own_fork, "compact": _own_compact}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, op = case, case["op"]
    if op == "prefix":
        B, H, P = c["B"], c["H"], c["shared"]
        mine = B * (c["own"] / 2.0)                       # lengths are uniform over [0, own]
        return {"bytes": (P + mine) * 1024 + 2 * B * H * 1024 + 4 * B * H + 4 * ((P + mine) / c["rpp"]),
                "flops": 4.0 * D * H * (B * P + mine)}
    if op == "window":
        B, H, W, S = c["B"], c["H"], c["window"], c["sink"]
        before = (c["ctx"] + 1) / 2.0 if c["ctx"] and B > 1 else c["ctx"]  # lengths are uniform over [1, ctx]
        rows = seen = 0.0
        for q in _chunks(c):
            rows += q + min(before, W + S)                # tokens that a window or a sink reaches
            short = min(max(0.0, W + S - before), q)      # the first tokens see less than a whole window
            seen += q * (W + S) - short * short / 2.0
        T = sum(_chunks(c))
        return {"bytes": rows * 1024 + 2 * T * H * 1024 + 4 * T * H + 4 * rows / c["rpp"], "flops": 4.0 * D * H * seen}
    page = 2.0 * sum(POOLS)
    if op == "fork":
        width, F = c["tokens"] // 64 + 1, c["children"]
        return {"bytes": 2 * F * page + 4.0 * width * (c["parents"] + F) + 8.0 * c["pages"], "flops": 0}
    used = max(1, int(c["pages"] * c["used"]))
    moved = used * (1 - used / c["pages"])                # pages in use that lie behind the first `used`
    return {"bytes": 2 * moved * page + 8.0 * (used + c["B"]) + 8.0 * c["pages"], "flops": 0}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    return {"prefix": _exact_prefix, "window": _exact_window, "fork": _exact_fork,
            "compact": _exact_compact}[case["op"]](case, seed)


def _attend64(q, kv, seen=None):
    """q [..., 512], kv [n, 512], seen broadcast over the rows of q: softmax(scale q kv^T) kv, and its lse."""
    x = SCALE * (q @ kv.t())
    if seen is not None:
        x = torch.where(seen, x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse.unsqueeze(-1)) @ kv, lse


def _rows64(s, b, lo, hi):
    rpp = s["case"]["rpp"]
    pages = s["table"][b].tolist()
    at = [pages[j // rpp] * rpp + j % rpp for j in range(lo, hi)]
    return s["pool"].index_select(0, torch.tensor(at, dtype=torch.int64, device="cuda")).double()


def _exact_prefix(c, seed):
    s = _prepare_prefix(c, seed)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["n_rows"].tolist()):
        out[b], lse[b] = _attend64(s["q"][b].double(), _rows64(s, b, 0, n))
    return {"out": out, "lse": lse}


def _exact_window(c, seed):
    s = _prepare_window(c, seed)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    at, lens = s["offsets"].tolist(), s["n_tokens"].tolist()
    for b in range(c["B"]):
        for t0 in range(at[b], at[b + 1], 256):
            t1 = min(t0 + 256, at[b + 1])
            p0 = lens[b] - (at[b + 1] - t0)
            p1 = p0 + (t1 - t0)
            lo = max(p0 - c["window"] + 1, 0)
            sinks = min(c["sink"], lo)
            kv = _rows64(s, b, lo, p1)
            if sinks:
                kv = torch.cat([_rows64(s, b, 0, sinks), kv])
            key = torch.cat([torch.arange(sinks), torch.arange(lo, p1)]).cuda()
            pos = torch.arange(p0, p1, device="cuda").view(-1, 1, 1)
            seen = (key <= pos) & ((key > pos - c["window"]) | (key < c["sink"]))
            out[t0:t1], lse[t0:t1] = _attend64(s["q"][t0:t1].double(), kv, seen)
    return {"out": out, "lse": lse}


def _exact_fork(c, seed):
    s = _prepare_fork(c, seed)
    table, refs, n_tokens = s["table"].tolist(), s["refs"].tolist(), s["n_tokens"].tolist()
    free = [i for i, r in enumerate(refs) if r == 0]
    width = len(table[0])
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        n = n_tokens[a]
        table[b] = table[a][: n // 64] + [-1] * (width - n // 64)
        for p in table[a][: n // 64]:
            refs[p] += 1
        if n % 64:
            table[b][n // 64] = free.pop(0)
            refs[table[b][n // 64]] = 1
        n_tokens[b] = n
    t = lambda x, d: torch.tensor(x, dtype=d)  # noqa: E731
    return {"table": t(table, torch.int32), "refs": t(refs, torch.int32), "n_tokens": t(n_tokens, torch.int64),
            "pools": None}


def _exact_compact(c, seed):
    s = _prepare_compact(c, seed)
    refs = s["refs"].tolist()
    n = sum(r > 0 for r in refs)
    holes = [i for i in range(n) if refs[i] == 0]
    to = {}
    for i in range(n, len(refs)):
        if refs[i]:
            to[i] = holes[len(to)]
            refs[to[i]], refs[i] = refs[i], 0
    table = [[to.get(p, p) for p in row] for row in s["table"].tolist()]
    return {"table": torch.tensor(table, dtype=torch.int32), "refs": torch.tensor(refs, dtype=torch.int32),
            "n_used": torch.tensor([n], dtype=torch.int64), "pools": None}
