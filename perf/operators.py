"""Measured cases of the operators around the int8 KV cache.

Three groups of operators, each with its plain form in elementary torch
operations (``own`` false) and the library's own call (``own`` true):

* ``diff``    differential decode attention over the int8 cache, contiguous or
              paged, M draft columns: (softmax_1 - lam * softmax_2) V per pair
              of heads;
* ``norm``    residual addition, root-mean-square norm, and an output held in
              8 bits with scales (int8 or e4m3, a scale per row or per 128
              channels);
* ``fork``, ``turnover``, ``compact``   the pages of a cache: copy-on-write
              forks with their page copies, retiring and admitting sequences,
              and compaction with its page moves.
"""

import math

import numpy as np
import torch

own = False

D = 128          # channels of a cache row
DEV = "cuda"


# ------------------------------------------------------------------ cases

def _diff(name, B, M, Hq, Hkv, lo, hi, page, per_row):
    return {"name": name, "op": "diff", "B": B, "M": M, "Hq": Hq, "Hkv": Hkv, "lo": lo, "hi": hi,
            "page": page, "per_row": per_row}


def _norm(name, rows, d, dtype, residual, out, group):
    return {"name": name, "op": "norm", "rows": rows, "d": d, "dtype": dtype, "residual": residual,
            "out": out, "group": group}


def _pages(name, op, slots, max_pages, n_pages, page, Hkv, n, fill):
    return {"name": name, "op": op, "slots": slots, "max_pages": max_pages, "n_pages": n_pages,
            "page": page, "Hkv": Hkv, "n": n, "fill": fill}


def listed():
    return [
        # one chat, just past 256 keys, 8 query and 2 kv heads: latency alone
        _diff("diff_one_chat", 1, 1, 8, 2, 257, 257, 0, False),
        # a serving batch of ragged contexts over shuffled 64-row pages
        _diff("diff_serving_paged", 64, 1, 32, 4, 512, 32768, 64, False),
        # speculative verify: 5 draft columns, a lam of its own for every row
        _diff("diff_verify", 16, 5, 32, 4, 1024, 4096, 0, True),
        # the norm in front of a projection in a decode step of 16 sequences
        _norm("norm_step", 16, 2048, "bfloat16", True, "int8", 0),
        # the same norm over a long prompt
        _norm("norm_prompt", 8192, 4096, "bfloat16", True, "int8", 0),
        # the norm of each 256-wide head of the attention's float32 output,
        # rows of a serving batch, for an e4m3 product with 128-channel scales
        _norm("norm_heads", 16384, 256, "float32", False, "e4m3", 128),
        # two branches from each of a few sequences (parallel sampling)
        _pages("fork_few", "fork", 64, 128, 4096, 64, 4, 8, 0.5),
        # every sequence of a large batch branches (tree search)
        _pages("fork_batch", "fork", 1024, 512, 65536, 64, 4, 512, 0.5),
        # a step of a small server: a few sequences end, others start
        _pages("turnover_few", "turnover", 64, 128, 4096, 64, 4, 8, 0.5),
        # a large server turns over a quarter of its slots
        _pages("turnover_batch", "turnover", 2048, 512, 262144, 64, 4, 512, 0.5),
        # compaction of a small, half empty pool of 32-row pages
        _pages("compact_small", "compact", 64, 96, 2048, 32, 2, 0, 0.45),
        # compaction of a large pool: thousands of pages move
        _pages("compact_large", "compact", 512, 512, 32768, 64, 4, 0, 0.6),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["diff", "diff", "norm", "norm", "fork", "turnover", "compact"])
    if op == "diff":
        M = rng.randint(1, 8)
        g = rng.choice([x for x in (1, 2, 3, 4, 5, 6, 7, 8, 16) if x * M <= 64])
        Hkv = rng.choice([2, 4, 6, 8])
        B = log_int(1, 96)
        # at most the keys and the score rows of the largest listed case
        top = min(131072, 64 * 32768 * 4 // (B * Hkv), 64 * 32768 * 32 // (B * Hkv * g * M))
        lo = log_int(1, max(2, top // 2))
        hi = max(lo, log_int(lo, max(lo + 1, top)))
        hi = min(hi, max(lo, 7800 * 64 * 4 // (B * Hkv)))
        return {k: v for k, v in _diff("", B, M, g * Hkv, Hkv, lo, hi,
                                       rng.choice([0, 32, 64, 128, 256]), rng.random() < 0.5).items()
                if k != "name"}
    if op == "norm":
        d = log_int(1, 16384)
        group = rng.choice([0, 128])
        if group:
            d = max(128, d // 128 * 128)
        rows = log_int(1, max(2, min(65536, 8192 * 4096 // d)))
        case = _norm("", rows, d, rng.choice(["bfloat16", "float16", "float32"]),
                     rng.random() < 0.6, rng.choice(["int8", "int8", "e4m3"]), group)
        return {k: v for k, v in case.items() if k != "name"}
    slots = log_int(3, 1500)
    max_pages = log_int(2, 600)
    page = rng.choice([32, 64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    fill = round(rng.uniform(0.1, 0.65), 2)
    top = min(200000, 32768 * 64 * 4 // (page * Hkv))
    n_pages = log_int(4 * slots, max(4 * slots + 1, top))
    case = _pages("", op, slots, max_pages, n_pages, page, Hkv,
                  0 if op == "compact" else log_int(1, max(2, slots // 3)), fill)
    return {k: v for k, v in case.items() if k != "name"}


# ---------------------------------------------------------------- prepare

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _contexts(case, seed):
    r = np.random.default_rng(seed * 7919 + 1)
    lo, hi = case["lo"], case["hi"]
    ctx = np.clip(np.floor(np.exp(r.uniform(math.log(lo), math.log(hi + 1), case["B"]))), lo, hi)
    return ctx.astype(np.int32), r


def _prepare_diff(case, seed):
    ctx, r = _contexts(case, seed)
    B, M, Hq, Hkv, page = (case[k] for k in ("B", "M", "Hq", "Hkv", "page"))
    keys = ctx.astype(np.int64) + M - 1
    g = _gen(seed)
    s = {"op": "diff", "M": M, "page": page, "max_ctx": int(ctx.max())}
    if page:
        pages = (keys + page - 1) // page
        order = r.permutation(int(pages.sum()) + 3).astype(np.int32)
        table = np.full((B, int(pages.max())), -1, np.int32)
        at = np.concatenate([[0], np.cumsum(pages)])
        for b in range(B):
            table[b, :pages[b]] = order[at[b]:at[b + 1]]
        cap = len(order) * page
        s["table"] = torch.from_numpy(table).to(DEV)
    else:
        gaps = r.integers(0, 4, B)
        start = np.concatenate([[0], np.cumsum(keys + gaps)[:-1]])
        cap = int((keys + gaps).sum())
        s["row_start"] = torch.from_numpy(start.astype(np.int64)).to(DEV)
    s["ctx"] = torch.from_numpy(ctx).to(DEV)
    # int8 rows as absmax quantization of normal values leaves them, and the
    # scales of such rows
    for name in ("k", "v"):
        s[name] = torch.randint(-127, 128, (Hkv, cap, D), generator=g, device=DEV, dtype=torch.int8)
        s[name + "s"] = (torch.rand((Hkv, cap), generator=g, device=DEV) + 0.5) * (2.0 / 127)
    s["q"] = torch.randn((B, M, Hq, D), generator=g, device=DEV)
    H = Hq // 2
    shape = (B, M, H) if case["per_row"] else (H,)
    s["lam"] = 0.2 + 0.6 * torch.rand(shape, generator=g, device=DEV)
    return s


def _prepare_norm(case, seed):
    g = _gen(seed)
    rows, d = case["rows"], case["d"]
    t = getattr(torch, case["dtype"])
    gain = 1.0 + 4.0 * (torch.rand(d, generator=g, device=DEV) < 0.01)   # a few wide channels
    s = {"op": "norm", "eps": 1e-6, "group": case["group"], "out": case["out"],
         "x": (torch.randn((rows, d), generator=g, device=DEV) * gain).to(t),
         "w": (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(t), "res": None}
    if case["residual"]:
        s["res"] = (2.0 * torch.randn((rows, d), generator=g, device=DEV)).to(t)
        s["res_out"] = torch.empty_like(s["res"])
    return s


def _pool(case, seed):
    """A pool in use: slots with pages in shuffled order, some of them sharing
    the pages of a common prompt.  Returns table, refs, lens (rows held)."""
    r = np.random.default_rng(seed * 104729 + 3)
    S, mp, n, page = case["slots"], case["max_pages"], case["n_pages"], case["page"]
    want = max(1, int(n * case["fill"]))
    share = r.random(S)
    count = np.maximum(1, np.floor(share / share.sum() * want).astype(np.int64))
    count = np.minimum(count, mp)
    if case["op"] != "compact" and S > 1:
        count[S // 2:] = np.minimum(count[S // 2:], max(1, mp // 2))
    while count.sum() > n - 1:                       # tiny pools: leave a page free
        count[np.argmax(count)] -= 1
        if count.max() <= 1:
            break
    order = r.permutation(n).astype(np.int32)
    table = np.full((S, mp), -1, np.int32)
    at = 0
    for i in range(S):
        c = int(min(count[i], n - at))
        table[i, :c] = order[at:at + c]
        at += c
        if c and i % 4 == 3 and count[i - 1]:        # shares its neighbour's first page
            table[i, 0] = table[i - 1, 0]
    used = table[table >= 0]
    refs = np.bincount(used, minlength=n).astype(np.int32)
    held = (table >= 0).sum(1)
    lens = np.maximum(0, held * page - r.integers(0, page, S) * (held > 0))
    return table, refs, lens.astype(np.int32), r


def _prepare_pages(case, seed):
    table, refs, lens, r = _pool(case, seed)
    S, page, n = case["slots"], case["page"], case["n_pages"]
    s = {"op": case["op"], "page": page,
         "table": torch.from_numpy(table).to(DEV), "refs": torch.from_numpy(refs).to(DEV)}
    if case["op"] != "turnover":
        g = _gen(seed)
        for name in ("k", "v"):
            s[name] = torch.randint(-127, 128, (case["Hkv"], n * page, D), generator=g, device=DEV,
                                    dtype=torch.int8)
            s[name + "s"] = torch.rand((case["Hkv"], n * page), generator=g, device=DEV)
    if case["op"] == "fork":
        # children are slots whose sequence ended, parents the others; parents
        # may branch more than once
        m = min(case["n"], S // 2)
        slots = r.permutation(S)
        child, parent = slots[:m], slots[m:][r.integers(0, S - m, m)]
        s["children"] = torch.from_numpy(child.astype(np.int32)).to(DEV)
        s["parents"] = torch.from_numpy(parent.astype(np.int32)).to(DEV)
        s["lens"] = torch.from_numpy(lens[parent].astype(np.int32)).to(DEV)
    if case["op"] == "turnover":
        m = min(case["n"], S)
        slots = r.permutation(S)[:m]
        s["seqs"] = torch.from_numpy(slots.astype(np.int32)).to(DEV)
        free = int((refs == 0).sum())
        most = max(1, min(case["max_pages"], free // m)) * page      # the pool has room for all
        s["lens"] = torch.from_numpy(r.integers(1, most + 1, m).astype(np.int32)).to(DEV)
    return s


def prepare(case, seed):
    if case["op"] == "diff":
        return _prepare_diff(case, seed)
    if case["op"] == "norm":
        return _prepare_norm(case, seed)
    return _prepare_pages(case, seed)


# ------------------------------------------------------------ plain forms

def _quantize_rows(x):
    a = x.abs().amax(-1, keepdim=True)
    scale = a / torch.full_like(a, 127.0)
    q = torch.where(scale > 0, torch.round(x / torch.where(scale > 0, scale, 1.0)), 0.0)
    return q.clamp(-127, 127), scale


def _plain_diff(s):
    q, k, v, ctx, lam, M, page = (s[n] for n in ("q", "k", "v", "ctx", "lam", "M", "page"))
    B, _, Hq, _ = q.shape
    Hkv = k.shape[0]
    g, P = Hq // Hkv, Hkv // 2
    T = s["max_ctx"] + M - 1
    t = torch.arange(T, device=q.device)
    last = (ctx.long() + M - 1)[:, None]
    tc = torch.minimum(t[None], last - 1)                              # stay inside the sequence
    if page:
        rows = s["table"].long().gather(1, tc // page) * page + tc % page
    else:
        rows = s["row_start"][:, None] + tc
    q8, qs = _quantize_rows(q)
    # head 2i + a reads key plane 2 (i // g) + a; [B, P, 2 (map), M, g, ...]
    q8 = q8.view(B, M, P, g, 2, D).permute(0, 2, 4, 1, 3, 5).reshape(B, P, 2, M * g, D)
    qs = qs.view(B, M, P, g, 2, 1).permute(0, 2, 4, 1, 3, 5).reshape(B, P, 2, M * g, 1)
    kf = k[:, rows].float().view(P, 2, B, T, D).permute(2, 0, 1, 3, 4)  # [B, P, 2, T, D]
    S = q8 @ kf.transpose(-1, -2)                                       # integers below 2^24
    del kf
    ks = s["ks"][:, rows].view(P, 2, B, 1, T).permute(2, 0, 1, 3, 4)
    x = S * (qs * ks)
    del S
    x = x * torch.full_like(qs, 1.0 / math.sqrt(D))
    seen = t[None, None] < ctx[:, None, None] + torch.arange(M, device=q.device)[None, :, None]
    seen = seen[:, :, None].expand(B, M, g, T).reshape(B, 1, 1, M * g, T)
    x = x.masked_fill(~seen, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    del x
    p = p / p.sum(-1, keepdim=True)
    lam_rows = lam.expand(B, M, Hq // 2).view(B, M, P, g).permute(0, 2, 1, 3).reshape(B, P, M * g, 1)
    w = p[:, :, 0] - lam_rows * p[:, :, 1]                              # [B, P, M g, T]
    del p
    vf = v[:, rows].float() * s["vs"][:, rows][..., None]               # [Hkv, B, T, D]
    vf = vf.view(P, 2, B, T, D).permute(2, 0, 3, 1, 4).reshape(B, P, T, 2 * D)
    o = w @ vf
    return o.view(B, P, M, g, 2 * D).permute(0, 2, 1, 3, 4).reshape(B, M, Hq // 2, 2 * D)


def _plain_norm(s):
    t = s["x"].dtype
    h = s["x"].float()
    res = None
    if s["res"] is not None:
        res = (h + s["res"].float()).to(t)
        h = res.float()
    r = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + s["eps"])
    rows, d = h.shape
    gs = s["group"] or d
    z = (h * s["w"].float()).view(rows, d // gs, gs)
    a = z.abs().amax(-1, keepdim=True)
    top = 127.0 if s["out"] == "int8" else 448.0
    s0 = a / torch.full_like(a, top)
    u = z / torch.where(s0 > 0, s0, 1.0)
    u = torch.where(s0 > 0, u, 0.0)
    if s["out"] == "int8":
        c = torch.round(u).clamp(-127, 127)
    else:
        c = u.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    y = (c * (s0 * r.view(rows, 1, 1))).view(rows, d)
    return {"y": y} if res is None else {"y": y, "residual": res}


def _plain_free(table, refs, seqs):
    seqs = seqs.long()
    rows = table[seqs]
    held = rows >= 0
    refs.scatter_add_(0, rows.clamp(min=0).long().view(-1), -held.to(torch.int32).view(-1))
    table[seqs] = -1


def _plain_take(refs, miss):
    """The lowest free pages for the true places of `miss`, in order."""
    free = torch.nonzero(refs == 0).view(-1)
    rank = torch.cumsum(miss.view(-1).long(), 0) - 1
    page = free[rank.clamp(min=0, max=max(0, free.numel() - 1))].view(miss.shape)
    refs.scatter_add_(0, page.view(-1), miss.to(torch.int32).view(-1))
    return page.to(torch.int32)


def _plain_reserve(table, refs, seqs, lens, page):
    seqs = seqs.long()
    rows = table[seqs]
    need = (lens.long() + page - 1) // page
    miss = (torch.arange(table.shape[1], device=table.device)[None] < need[:, None]) & (rows < 0)
    table[seqs] = torch.where(miss, _plain_take(refs, miss), rows)


def _plain_copy(s, src, dst):
    Hkv, cap, _ = s["k"].shape
    page = s["page"]
    at = torch.nonzero(src >= 0).view(-1)
    a, b = src[at].long(), dst[at].long()
    for name, width in (("k", page * D), ("v", page * D), ("ks", page), ("vs", page)):
        x = s[name].view(Hkv, cap // page, width)
        x[:, b] = x[:, a]


def _plain_fork(s):
    table, refs, page, lens = s["table"], s["refs"], s["page"], s["lens"].long()
    _plain_free(table, refs, s["children"])
    rows = table[s["parents"].long()]
    cols = torch.arange(table.shape[1], device=table.device)[None]
    full, tail = lens // page, lens % page > 0
    shared = cols < full[:, None]
    new = _plain_take(refs, tail)
    refs.scatter_add_(0, rows.clamp(min=0).long().view(-1), shared.to(torch.int32).view(-1))
    child = torch.where(shared, rows, -1)
    child = torch.where((cols == full[:, None]) & tail[:, None], new[:, None], child)
    last = rows.gather(1, full.clamp(max=table.shape[1] - 1)[:, None]).view(-1)
    src, dst = torch.where(tail, last, -1), torch.where(tail, new, -1)
    table[s["children"].long()] = child
    _plain_copy(s, src, dst)
    return src, dst


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    n = refs.numel()
    live = refs > 0
    n_live = live.sum()
    at = torch.arange(n, device=refs.device)
    holes = torch.nonzero(~live & (at < n_live)).view(-1)
    movers = torch.nonzero(live & (at >= n_live)).view(-1)
    to = at.clone()
    to[movers] = holes
    table_out = torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table)
    refs_out = refs.clone()
    refs_out[holes] = refs[movers]
    refs_out[movers] = 0
    src = torch.full((max(1, n // 2),), -1, dtype=torch.int32, device=refs.device)
    dst = torch.full_like(src, -1)
    src[:movers.numel()] = movers.to(torch.int32)
    dst[:holes.numel()] = holes.to(torch.int32)
    counts = torch.stack([n_live.to(torch.int32), live[n_live:].sum().to(torch.int32)])
    _plain_copy(s, src, dst)
    return table_out, refs_out, src, dst, counts


# -------------------------------------------------------------------- run

def _kept(s, name, make):
    """A buffer that a serving program keeps between its steps."""
    if name not in s:
        s[name] = make()
    return s[name]


def _run_diff(s):
    if not own:
        return _plain_diff(s)
    import int8_kv_decode_gb300 as K
    q = s["q"]
    B, M, Hq, _ = q.shape
    ws = _kept(s, "ws", lambda: K.alloc_diff_workspace(B, M, Hq, s["max_ctx"], q.device))
    out = _kept(s, "out", lambda: torch.empty((B, M, Hq // 2, 2 * D), device=q.device))
    if s["page"]:
        return K.decode_diff_paged(q, s["k"], s["ks"], s["v"], s["vs"], s["table"], s["page"], s["ctx"],
                                   s["max_ctx"], s["lam"], out=out, workspace=ws)
    return K.decode_diff(q, s["k"], s["ks"], s["v"], s["vs"], s["row_start"], s["ctx"], s["max_ctx"],
                         s["lam"], out=out, workspace=ws)


def _run_norm(s):
    if not own:
        return _plain_norm(s)
    import int8_kv_decode_gb300 as K
    x = s["x"]
    rows, d = x.shape
    groups = d // s["group"] if s["group"] else 1
    t = torch.int8 if s["out"] == "int8" else torch.float8_e4m3fn
    out = _kept(s, "out_q", lambda: torch.empty((rows, d), dtype=t, device=x.device))
    scale = _kept(s, "out_scale", lambda: torch.empty((rows, groups), device=x.device))
    K.rms_norm_quant(x, s["w"], residual=s["res"], residual_out=s.get("res_out"), eps=s["eps"],
                     group=s["group"], out=out, out_scale=scale)
    # the values that the 8-bit codes stand for
    c = out if t == torch.int8 else out.float()
    y = (c.view(rows, groups, d // groups) * scale[:, :, None]).view(rows, d)
    return {"y": y} if s["res"] is None else {"y": y, "residual": s["res_out"]}


def _page_workspace(s, K):
    return _kept(s, "ws", lambda: K.alloc_page_workspace(s["table"].shape[0], s["refs"].numel(),
                                                         s["table"].device))


def _run_fork(s):
    if own:
        import int8_kv_decode_gb300 as K
        ws = _page_workspace(s, K)
        src, dst = K.fork_sequences(s["table"], s["refs"], s["parents"], s["children"], s["lens"],
                                    s["page"], workspace=ws)
        K.copy_pages(s["k"], s["ks"], s["v"], s["vs"], src, dst, s["page"], workspace=ws)
    else:
        src, dst = _plain_fork(s)
    return {"table": s["table"], "refs": s["refs"], "src": src, "dst": dst,
            "k": s["k"], "ks": s["ks"], "v": s["v"], "vs": s["vs"]}


def _run_turnover(s):
    if own:
        import int8_kv_decode_gb300 as K
        ws = _page_workspace(s, K)
        K.free_sequences(s["table"], s["refs"], s["seqs"], workspace=ws)
        K.reserve_pages(s["table"], s["refs"], s["seqs"], s["lens"], s["page"], workspace=ws)
    else:
        _plain_free(s["table"], s["refs"], s["seqs"])
        _plain_reserve(s["table"], s["refs"], s["seqs"], s["lens"], s["page"])
    return {"table": s["table"], "refs": s["refs"]}


def _run_compact(s):
    if own:
        import int8_kv_decode_gb300 as K
        ws = _page_workspace(s, K)
        table, refs, src, dst, counts = K.compact_pages(s["table"], s["refs"], workspace=ws)
        K.copy_pages(s["k"], s["ks"], s["v"], s["vs"], src, dst, s["page"], count=counts[1:],
                     workspace=ws)
    else:
        table, refs, src, dst, counts = _plain_compact(s)
    return {"table": table, "refs": refs, "src": src, "dst": dst, "counts": counts,
            "k": s["k"], "ks": s["ks"], "v": s["v"], "vs": s["vs"]}


def run(state):
    return {"diff": _run_diff, "norm": _run_norm, "fork": _run_fork, "turnover": _run_turnover,
            "compact": _run_compact}[state["op"]](state)


# ------------------------------------------------------------------- work

def work(case):
    if case["op"] == "diff":
        ctx, _ = _contexts(case, 0)
        M, Hq, Hkv, B = case["M"], case["Hq"], case["Hkv"], case["B"]
        keys = float((ctx.astype(np.int64) + M - 1).sum())
        seen = float((ctx.astype(np.int64) * M + M * (M - 1) // 2).sum())
        io = 2 * B * M * Hq * D * 4 + (B * M * Hq // 2 if case["per_row"] else Hq // 2) * 4
        table = 4 * sum(-(-(int(c) + M - 1) // case["page"]) for c in ctx) if case["page"] else 0
        # QK: D products a key and head; PV: 2 D for the difference of a pair's maps
        return {"bytes": keys * Hkv * (2 * D + 8) + io + table + B * 12,
                "flops": seen * (Hq * D * 2 + Hq // 2 * 2 * D * 2 + Hq * 4)}
    if case["op"] == "norm":
        n, e = case["rows"] * case["d"], 4 if case["dtype"] == "float32" else 2
        groups = case["d"] // case["group"] if case["group"] else 1
        # codes and scales are written, and read once for the values returned
        return {"bytes": n * (e * (3 if case["residual"] else 1) + 1 + 1 + 4)
                + 2 * case["rows"] * groups * 4 + case["d"] * e, "flops": n * 8}
    page_bytes = 2 * case["Hkv"] * case["page"] * (D + 4)
    table, refs, lens, _ = _pool(case, 0)
    if case["op"] == "turnover":
        n = min(case["n"], case["slots"])
        return {"bytes": 4.0 * (2 * n * table.shape[1] + 2 * n) + 4.0 * refs.size, "flops": refs.size}
    if case["op"] == "fork":
        n = min(case["n"], case["slots"] // 2)
        return {"bytes": 2.0 * n * page_bytes + 4.0 * (3 * n * table.shape[1] + refs.size),
                "flops": refs.size}
    live = int((refs > 0).sum())
    moved = int((refs[live:] > 0).sum())
    return {"bytes": 2.0 * moved * page_bytes + 8.0 * table.size + 8.0 * refs.size + 4.0 * refs.size,
            "flops": refs.size + table.size}


# ------------------------------------------------------------------ exact

def _exact_diff(case, seed):
    s = _prepare_diff(case, seed)
    B, M, Hq, Hkv, page = (case[k] for k in ("B", "M", "Hq", "Hkv", "page"))
    g, H = Hq // Hkv, Hq // 2
    ctx = s["ctx"].cpu().numpy()
    if float((ctx.astype(np.float64) + M).sum()) * M * Hq * 6 * D > 6e12:
        return None
    out = torch.empty((B, M, H, 2 * D), dtype=torch.float64, device=DEV)
    # the query codes are defined by float32 divisions, rounded half to even
    q = s["q"].cpu().numpy()
    qs = (np.abs(q).max(-1) / np.float32(127)).astype(np.float32)
    q8 = np.clip(np.rint(q / np.where(qs > 0, qs, 1)[..., None]), -127, 127)
    q8 = torch.from_numpy(np.where(qs[..., None] > 0, q8, 0).astype(np.float64)).to(DEV)
    qs = torch.from_numpy(qs.astype(np.float64)).to(DEV)
    lam = s["lam"].double().expand(B, M, H)
    for b in range(B):
        n = int(ctx[b]) + M - 1
        if page:
            pages = s["table"][b, :(n + page - 1) // page].long()
            rows = (pages[:, None] * page + torch.arange(page, device=DEV)[None]).view(-1)[:n]
        else:
            rows = torch.arange(n, device=DEV) + s["row_start"][b]
        for pair in range(Hkv // 2):
            value = torch.cat([s["v"][2 * pair + c][rows].double() * s["vs"][2 * pair + c][rows].double()[:, None]
                               for c in (0, 1)], 1)
            heads = torch.arange(pair * g, pair * g + g, device=DEV)
            maps = []
            for a in (0, 1):
                key = s["k"][2 * pair + a][rows].double() * s["ks"][2 * pair + a][rows].double()[:, None]
                query = q8[b][:, 2 * heads + a] * qs[b][:, 2 * heads + a, None]      # [M, g, D]
                score = query @ key.t() / math.sqrt(D)
                for j in range(M):
                    score[j, :, int(ctx[b]) + j:] = -math.inf
                maps.append(torch.softmax(score, -1) @ value)
            out[b, :, pair * g:pair * g + g] = maps[0] - lam[b][:, pair * g:pair * g + g, None] * maps[1]
    return out


def _exact_norm(case, seed):
    s = _prepare_norm(case, seed)
    x = s["x"].float().cpu().numpy()
    res = None
    if s["res"] is not None:
        total = torch.from_numpy(x.astype(np.float64) + s["res"].cpu().double().numpy())
        res = total.to(torch.float32).to(s["x"].dtype)     # float32 sums of 16-bit or float32 values
        x = res.float().numpy()
    w = s["w"].float().cpu().numpy()
    rms = np.sqrt((x.astype(np.float64) ** 2).mean(-1) + s["eps"])
    # the codes are defined on the float32 products and divisions
    z = (x * w).reshape(x.shape[0], -1, s["group"] or x.shape[1])
    top = np.float32(127 if s["out"] == "int8" else 448)
    s0 = (np.abs(z).max(-1, keepdims=True) / top).astype(np.float32)
    u = np.where(s0 > 0, z / np.where(s0 > 0, s0, 1), 0).astype(np.float32)
    if s["out"] == "int8":
        c = np.clip(np.rint(u), -127, 127).astype(np.float64)
    else:
        a = np.abs(u.astype(np.float64))
        step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(a, 1e-30))), -6) - 3)
        c = np.sign(u) * np.minimum(np.rint(a / step) * step, 448.0)
    y = (c * s0.astype(np.float64) / rms[:, None, None]).reshape(x.shape)
    y = torch.from_numpy(y)
    return {"y": y} if res is None else {"y": y, "residual": res.double()}


def _exact_pages(case, seed):
    """The float scales of the pool after the copies (the rest are whole
    numbers), from a page-by-page account on the host."""
    if case["op"] == "turnover":
        return None
    s = _prepare_pages(case, seed)
    table, refs, page = s["table"].cpu().numpy(), s["refs"].cpu().numpy(), s["page"]
    moves = []
    if case["op"] == "fork":
        children, parents, lens = (s[n].cpu().numpy() for n in ("children", "parents", "lens"))
        for c in children:
            for e in table[c][table[c] >= 0]:
                refs[e] -= 1
        free = iter(np.flatnonzero(refs == 0))
        for p, n in zip(parents, lens):
            if n % page:
                moves.append((table[p][n // page], next(free)))
    else:
        live = int((refs > 0).sum())
        moves = list(zip(np.flatnonzero(refs[live:] > 0) + live, np.flatnonzero(refs[:live] == 0)))
    out = {}
    for name in ("ks", "vs"):
        x = s[name].double().cpu().numpy()
        y = x.copy()
        for a, b in moves:
            y[:, b * page:(b + 1) * page] = x[:, a * page:(a + 1) * page]
        out[name] = torch.from_numpy(y)
    return out


def exact(case, seed):
    if case["op"] == "diff":
        return _exact_diff(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, seed)
    return _exact_pages(case, seed)
