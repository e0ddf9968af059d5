"""Measured cases of the operators on a cache whose 8-bit rows share a scale per
block of tokens and head.

Four operators, each with its plain form in elementary torch operations (``own``
false) and the library's own call (``own`` true):

* ``rope``    rotary positions of heads: the two layouts, all or part of the head;
* ``write``   new K and V rows into the paged cache (K rotated, one scale per block
              and head, the rows already in a block re-scaled where it grows), the
              queries rotated in the same call, and the touched blocks read back;
* ``read``    rows of sequences out of the paged cache, as 16- or 32-bit values;
* ``attend``  decode attention over that cache, M draft columns.
"""

import math

import numpy as np
import torch

own = False

D = 128          # channels of a head
DEV = "cuda"


# ------------------------------------------------------------------ cases

def _rope(name, rows, heads, dtype, out, rot, interleaved, positions):
    return {"name": name, "op": "rope", "rows": rows, "heads": heads, "dtype": dtype, "out": out,
            "rot": rot, "interleaved": interleaved, "positions": positions}


def _write(name, B, lo, hi, held, Hq, Hkv, dtype, code, block, page, rot, interleaved):
    return {"name": name, "op": "write", "B": B, "lo": lo, "hi": hi, "held": held, "Hq": Hq, "Hkv": Hkv,
            "dtype": dtype, "code": code, "block": block, "page": page, "rot": rot,
            "interleaved": interleaved}


def _read(name, B, lo, hi, Hkv, code, out, block, page):
    return {"name": name, "op": "read", "B": B, "lo": lo, "hi": hi, "Hkv": Hkv, "code": code, "out": out,
            "block": block, "page": page}


def _attend(name, B, M, Hq, Hkv, lo, hi, dtype, code, block, page):
    return {"name": name, "op": "attend", "B": B, "M": M, "Hq": Hq, "Hkv": Hkv, "lo": lo, "hi": hi,
            "dtype": dtype, "code": code, "block": block, "page": page}


def listed():
    return [
        # the queries and keys of one decode step of 16 sequences
        _rope("rope_step", 16, 36, "bfloat16", "bfloat16", 128, False, 32768),
        # those of a long prompt; the row-scaled cache's decode takes float32
        _rope("rope_prompt", 8192, 36, "bfloat16", "float32", 128, False, 32768),
        # half of each head, neighbouring channels in pairs, positions far out
        _rope("rope_far_part", 2000, 32, "float16", "float16", 64, True, 131072),
        # a decode step of a serving batch: one row for each of 64 sequences
        _write("write_step", 64, 1, 1, 8192, 32, 4, "bfloat16", "int8", 32, 64, 128, False),
        # the draft rows of a speculative step, e4m3 codes
        _write("write_drafts", 16, 5, 5, 4096, 32, 4, "float16", "e4m3", 64, 64, 128, False),
        # ragged prompts written at once, some of them behind a cached prefix
        _write("write_prompts", 7, 300, 2500, 1000, 32, 4, "bfloat16", "int8", 32, 64, 128, False),
        # one short prefix read back for a prompt that goes on
        _read("read_prefix", 1, 700, 700, 4, "int8", "bfloat16", 32, 64),
        # the contexts of a batch, for attention kernels on 16-bit rows
        _read("read_contexts", 24, 2048, 16384, 4, "e4m3", "bfloat16", 64, 64),
        # one chat, just past 256 keys, 8 query and 2 kv heads: latency alone
        _attend("attend_one_chat", 1, 1, 8, 2, 257, 257, "bfloat16", "int8", 32, 32),
        # a serving batch of ragged contexts over shuffled 64-row pages
        _attend("attend_serving", 64, 1, 32, 4, 512, 32768, "bfloat16", "int8", 32, 64),
        # speculative verify: 5 draft columns of 8 heads on each kv head
        _attend("attend_verify", 16, 5, 32, 4, 1024, 4096, "float16", "e4m3", 64, 64),
        # two long documents, float32 queries as the row-scaled cache takes them
        _attend("attend_long", 2, 1, 32, 4, 120000, 131072, "float32", "int8", 128, 128),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def pages():
        block = rng.choice([32, 64, 128])
        return block, rng.choice([p for p in (32, 64, 128, 256) if p >= block])

    op = rng.choice(["rope", "write", "write", "read", "attend", "attend", "attend"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    code = rng.choice(["int8", "e4m3"])
    rot = rng.choice([128, 128, 96, 64, 32, 8])
    if op == "rope":
        heads = rng.choice([1, 3, 8, 10, 36, 40, 64])
        case = _rope("", log_int(1, 8192 * 36 // heads), heads, dtype, rng.choice([dtype, "float32"]), rot,
                     rng.random() < 0.5, log_int(64, 131072))
    elif op == "write":
        block, page = pages()
        Hkv = rng.choice([1, 2, 4, 6, 8])
        Hq = Hkv * rng.choice([1, 4, 7, 8])
        B = log_int(1, 128)
        top = max(1, 8192 * 40 // (B * (Hq + 2 * Hkv)))
        lo = log_int(1, top)
        case = _write("", B, lo, log_int(lo, max(lo, top)), log_int(1, 8192), Hq, Hkv, dtype, code, block,
                      page, rot, rng.random() < 0.5)
    elif op == "read":
        block, page = pages()
        Hkv = rng.choice([1, 2, 4, 6, 8])
        B = log_int(1, 64)
        top = max(1, 24 * 7000 * 4 // (B * Hkv))
        lo = log_int(1, top)
        case = _read("", B, lo, log_int(lo, max(lo, top)), Hkv, code, rng.choice([dtype, "bfloat16"]), block,
                     page)
    else:
        block, page = pages()
        M = rng.randint(1, 8)
        g = rng.choice([x for x in (1, 2, 3, 4, 5, 6, 7, 8, 16) if x * M <= 64])
        Hkv = rng.choice([1, 2, 4, 8])
        B = log_int(1, 96)
        # at most the keys and the score rows of the largest listed case
        top = min(131072, 64 * 32768 * 4 // (B * Hkv), 64 * 32768 * 32 // (B * Hkv * g * M))
        lo = log_int(1, max(2, top // 2))
        hi = max(lo, log_int(lo, max(lo + 1, top)))
        hi = min(hi, max(lo, 7800 * 64 * 4 // (B * Hkv)))
        case = _attend("", B, M, g * Hkv, Hkv, lo, hi, dtype, code, block, page)
    return {k: v for k, v in case.items() if k != "name"}


# ---------------------------------------------------------------- prepare

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _spread(case, seed):
    """Lengths of the sequences, and the rows that each holds before its first: the
    case's own, in an order of the seed's, with a generator for what else it decides."""
    r = np.random.default_rng([case["B"], case["lo"], case["hi"]])
    lo, hi = case["lo"], case["hi"]
    n = np.clip(np.floor(np.exp(r.uniform(math.log(lo), math.log(hi + 1), case["B"]))), lo, hi).astype(np.int64)
    start = np.zeros_like(n)
    if case["op"] == "read":
        start = r.integers(0, 40, len(n)) * (r.random(len(n)) < 0.5)
    if case["op"] == "write":
        held = np.floor(np.exp(r.uniform(0, math.log(case["held"] + 1), len(n)))).astype(np.int64)
        start = held * (r.random(len(n)) < (0.5 if hi > 64 else 0.95))
    r = np.random.default_rng(seed * 7919 + 1)
    order = r.permutation(len(n))
    return n[order], start[order], r


def _rope_table(n, rot):
    """cos and sin of every position, the angles in 64 bits (a program makes it once)."""
    freq = 500000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    angle = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], -1).float()


def _table(r, pages, spare=3):
    order = r.permutation(int(pages.sum()) + spare).astype(np.int32)
    table = np.full((len(pages), int(pages.max())), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(pages)])
    for b in range(len(pages)):
        table[b, :pages[b]] = order[at[b]:at[b + 1]]
    return table, len(order)


def _cache(s, case, n_pages, g):
    """A cache in use: normal values under a scale per block and head."""
    Hkv, cap = case["Hkv"], n_pages * case["page"]
    for name in ("k", "v"):
        x = torch.randn((Hkv, cap, D), generator=g, device=DEV)
        if case["code"] == "int8":
            s[name] = torch.round(x * 30).clamp(-127, 127).to(torch.int8)
        else:
            s[name] = (x * 105).clamp(-448, 448).to(torch.float8_e4m3fn)
        del x
        s[name + "s"] = (torch.rand((Hkv, cap // case["block"]), generator=g, device=DEV) + 0.5) \
            * (1 / 30 if case["code"] == "int8" else 1 / 105)
    s.update(page=case["page"], block=case["block"], code=case["code"])


def _spans(s, n, start):
    s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(DEV)
    s["start"] = torch.from_numpy(start.astype(np.int32)).to(DEV)
    s["rows"] = int(n.sum())


def _prepare_rope(case, seed):
    g = _gen(seed)
    n = case["positions"]
    x = torch.randn((case["rows"], case["heads"], D), generator=g, device=DEV)
    return {"op": "rope", "x": x.to(getattr(torch, case["dtype"])), "out": getattr(torch, case["out"]),
            "positions": torch.randint(0, n, (case["rows"],), generator=g, device=DEV, dtype=torch.int32),
            "table": _rope_table(n, case["rot"]), "interleaved": case["interleaved"]}


def _prepare_write(case, seed):
    n, start, r = _spread(case, seed)
    g = _gen(seed)
    s = {"op": "write", "interleaved": case["interleaved"]}
    table, n_pages = _table(r, -(-(start + n) // case["page"]))
    _cache(s, case, n_pages, g)
    s["table"] = torch.from_numpy(table).to(DEV)
    _spans(s, n, start)
    T, Hq, Hkv = s["rows"], case["Hq"], case["Hkv"]
    # the rows of one fused projection: queries, keys, values side by side, some
    # channels wider than the rest
    gain = 1.0 + 3.0 * (torch.rand(((Hq + 2 * Hkv), D), generator=g, device=DEV) < 0.02)
    qkv = (torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=DEV) * gain).to(getattr(torch, case["dtype"]))
    s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    s["rope"] = _rope_table(int((start + n).max()), case["rot"])
    # what the touched blocks hold afterwards
    first = start // case["block"] * case["block"]
    back = {}
    _spans(back, start + n - first, first)
    s["back"] = back
    return s


def _prepare_read(case, seed):
    n, start, r = _spread(case, seed)
    s = {"op": "read", "out": getattr(torch, case["out"])}
    table, n_pages = _table(r, -(-(start + n) // case["page"]))
    _cache(s, case, n_pages, _gen(seed))
    s["table"] = torch.from_numpy(table).to(DEV)
    _spans(s, n, start)
    return s


def _prepare_attend(case, seed):
    ctx, _, r = _spread(case, seed)
    M = case["M"]
    g = _gen(seed)
    s = {"op": "attend", "M": M, "max_ctx": int(ctx.max())}
    table, n_pages = _table(r, -(-(ctx + M - 1) // case["page"]))
    _cache(s, case, n_pages, g)
    s["table"] = torch.from_numpy(table).to(DEV)
    s["ctx"] = torch.from_numpy(ctx.astype(np.int32)).to(DEV)
    q = torch.randn((case["B"], M, case["Hq"], D), generator=g, device=DEV)
    s["q"] = q.to(getattr(torch, case["dtype"]))
    return s


def prepare(case, seed):
    return {"rope": _prepare_rope, "write": _prepare_write, "read": _prepare_read,
            "attend": _prepare_attend}[case["op"]](case, seed)


# ------------------------------------------------------------ plain forms

def _rotate(x, table, positions, interleaved):
    """Every product and sum in float32, one operation at a time."""
    h = table.shape[1]
    cs = table[positions.long()][:, None]                               # [T][1][h][2]
    c, s = cs[..., 0], cs[..., 1]
    x = x.float()
    y = x.clone()
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if interleaved else (x[..., :h], x[..., h:2 * h])
    lo, hi = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = lo, hi
    else:
        y[..., :h], y[..., h:2 * h] = lo, hi
    return y


def _plain_rope(s):
    return _rotate(s["x"], s["table"], s["positions"], s["interleaved"]).to(s["out"])


def _rows_of(s, spans):
    """Sequence, key position and physical row of every row of ragged spans."""
    T = spans["rows"]
    at = torch.arange(T, device=DEV)
    b = torch.searchsorted(spans["cu"].long(), at, right=True) - 1
    pos = spans["start"].long()[b] + at - spans["cu"].long()[b]
    return b, pos, s["table"].long()[b, pos // s["page"]] * s["page"] + pos % s["page"]


def _round_codes(u, code):
    if code == "int8":
        return torch.round(u).clamp(-127, 127).to(torch.int8)
    return u.clamp(-448, 448).to(torch.float8_e4m3fn)


def _bytes(x):
    return x.view(torch.uint8)


def _as_codes(x, code):
    return x.view(torch.int8 if code == "int8" else torch.float8_e4m3fn)


def _write_rows(s, name, x, b, pos, row):
    """x [T][Hkv][D] float32 into rows `row` of the cache `name`."""
    R, code, codes, scales = s["block"], s["code"], s[name], s[name + "s"]
    top = 127.0 if code == "int8" else 448.0
    x = x.transpose(0, 1)                                               # [Hkv][T][D]
    amax = x.abs().amax(-1)                                             # [Hkv][T]
    # the largest of the new rows of each block of the pool
    fresh = torch.zeros_like(scales).scatter_reduce_(
        1, (row // R).expand(x.shape[0], -1), amax, "amax")
    start = fresh / torch.full_like(fresh, top)
    # the blocks whose first rows stay: those of a sequence that goes on inside one
    first = s["start"].long()
    goes_on = (first % R != 0) & (s["cu"][1:] > s["cu"][:-1])
    kept = torch.nonzero(goes_on).view(-1)
    block = (s["table"].long()[kept, first[kept] // s["page"]] * s["page"] + first[kept] % s["page"]) // R
    old = scales[:, block]
    new = torch.maximum(old, start[:, block])
    lane = torch.arange(R, device=DEV)
    rows = block[:, None] * R + lane                                    # [kept][R]
    stays = (lane[None] < (first[kept] % R)[:, None])[None, :, :, None]
    was = _as_codes(_bytes(codes)[:, rows], code)                       # [Hkv][kept][R][D]
    f = torch.where(new > 0, old / torch.where(new > 0, new, 1.0), 1.0)[:, :, None, None]
    again = _round_codes(was.float() * f, code)
    grown = (new > old)[:, :, None, None]
    _bytes(codes)[:, rows] = torch.where(stays & grown, _bytes(again), _bytes(was))
    start[:, block] = new
    touched = torch.zeros_like(scales).index_fill_(1, row // R, 1.0) > 0
    scales.copy_(torch.where(touched, start, scales))
    # the new rows under their block's scale
    sc = scales[:, row // R][:, :, None]
    u = torch.where(sc > 0, x / torch.where(sc > 0, sc, 1.0), 0.0)
    _bytes(codes)[:, row] = _bytes(_round_codes(u, code))


def _read_rows(s, name, spans, out):
    _, _, row = _rows_of(s, spans)
    c = _as_codes(_bytes(s[name])[:, row], s["code"]).float()
    return (c * s[name + "s"][:, row // s["block"]][:, :, None]).transpose(0, 1).to(out).contiguous()


def _plain_write(s):
    b, pos, row = _rows_of(s, s)
    _write_rows(s, "k", _rotate(s["k_new"], s["rope"], pos, s["interleaved"]), b, pos, row)
    _write_rows(s, "v", s["v_new"].float(), b, pos, row)
    q = _rotate(s["q"], s["rope"], pos, s["interleaved"]).to(s["q"].dtype)
    return {"q": q, "k": _read_rows(s, "k", s["back"], torch.float32),
            "v": _read_rows(s, "v", s["back"], torch.float32), "ks": s["ks"], "vs": s["vs"]}


def _plain_read(s):
    return {"k": _read_rows(s, "k", s, s["out"]), "v": _read_rows(s, "v", s, s["out"])}


def _plain_attend(s):
    q, ctx, M, page = s["q"], s["ctx"], s["M"], s["page"]
    B, _, Hq, _ = q.shape
    Hkv = s["k"].shape[0]
    g = Hq // Hkv
    T = s["max_ctx"] + M - 1
    t = torch.arange(T, device=DEV)
    last = (ctx.long() + M - 1)[:, None]
    tc = torch.minimum(t[None], last - 1)                               # stay inside the sequence
    rows = s["table"].long().gather(1, tc // page) * page + tc % page   # [B][T]
    block = rows // s["block"]
    x = q.float().view(B, M, Hkv, g, D).permute(2, 0, 1, 3, 4).reshape(Hkv, B, M * g, D)
    kf = _as_codes(_bytes(s["k"])[:, rows], s["code"]).float()
    x = x @ kf.transpose(-1, -2)                                        # [Hkv][B][M g][T]
    del kf
    x = x * s["ks"][:, block][:, :, None]
    x = x * torch.full_like(x[..., :1], 1.0 / math.sqrt(D))
    seen = t[None, None] < ctx[:, None, None] + torch.arange(M, device=DEV)[None, :, None]
    x = x.masked_fill(~seen[:, :, None].expand(B, M, g, T).reshape(1, B, M * g, T), -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    del x
    p = p / p.sum(-1, keepdim=True)
    vf = _as_codes(_bytes(s["v"])[:, rows], s["code"]).float() * s["vs"][:, block][..., None]
    o = (p @ vf).view(Hkv, B, M, g, D).permute(1, 2, 0, 3, 4).reshape(B, M, Hq, D)
    return o.to(q.dtype)


# -------------------------------------------------------------------- run

def _kept(s, name, make):
    """A buffer that a serving program keeps between its steps."""
    if name not in s:
        s[name] = make()
    return s[name]


def _error_word(s):
    return _kept(s, "ws", lambda: torch.zeros(256, dtype=torch.uint8, device=DEV))


def _run_rope(s):
    if not own:
        return _plain_rope(s)
    import int8_kv_decode_gb300 as K
    out = _kept(s, "y", lambda: torch.empty(s["x"].shape, dtype=s["out"], device=DEV))
    return K.rope(s["x"], s["positions"], s["table"], interleaved=s["interleaved"], out=out)


def _run_write(s):
    if not own:
        return _plain_write(s)
    import int8_kv_decode_gb300 as K
    cache = (s["k"], s["ks"], s["v"], s["vs"])
    back = s["back"]
    q_out = _kept(s, "q_out", lambda: torch.empty(s["q"].shape, dtype=s["q"].dtype, device=DEV))
    shape = (back["rows"], s["k"].shape[0], D)
    k, v = (_kept(s, "back_" + n, lambda: torch.empty(shape, device=DEV)) for n in "kv")
    K.append_blocks(s["k_new"], s["v_new"], s["cu"], s["start"], *cache, s["table"], s["page"],
                    table=s["rope"], interleaved=s["interleaved"], q=s["q"], q_out=q_out,
                    workspace=_error_word(s))
    K.read_blocks(*cache, s["table"], s["page"], back["cu"], back["start"], back["rows"], out_k=k, out_v=v,
                  workspace=_error_word(s))
    return {"q": q_out, "k": k, "v": v, "ks": s["ks"], "vs": s["vs"]}


def _run_read(s):
    if not own:
        return _plain_read(s)
    import int8_kv_decode_gb300 as K
    shape = (s["rows"], s["k"].shape[0], D)
    k, v = (_kept(s, "out_" + n, lambda: torch.empty(shape, dtype=s["out"], device=DEV)) for n in "kv")
    K.read_blocks(s["k"], s["ks"], s["v"], s["vs"], s["table"], s["page"], s["cu"], s["start"], s["rows"],
                  out_k=k, out_v=v, workspace=_error_word(s))
    return {"k": k, "v": v}


def _run_attend(s):
    if not own:
        return _plain_attend(s)
    import int8_kv_decode_gb300 as K
    q = s["q"]
    B, M, Hq, _ = q.shape
    ws = _kept(s, "ws", lambda: K.alloc_blocks_workspace(B, M, Hq, s["max_ctx"], q.device))
    out = _kept(s, "out", lambda: torch.empty_like(q))
    return K.decode_blocks(q, s["k"], s["ks"], s["v"], s["vs"], s["table"], s["page"], s["ctx"],
                           s["max_ctx"], out=out, workspace=ws)


def run(state):
    return {"rope": _run_rope, "write": _run_write, "read": _run_read, "attend": _run_attend}[state["op"]](state)


# ------------------------------------------------------------------- work

def _size(dtype):
    return 4 if dtype == "float32" else 2


def work(case):
    if case["op"] == "rope":
        n = case["rows"] * case["heads"] * D
        table = 8 * min(case["rows"], case["positions"]) * (case["rot"] // 2)
        return {"bytes": float(n * (_size(case["dtype"]) + _size(case["out"])) + table + 4 * case["rows"]),
                "flops": 3.0 * case["rows"] * case["heads"] * case["rot"]}
    n, start, _ = _spread(case, 0)
    if case["op"] == "attend":
        M, Hq, Hkv, B = case["M"], case["Hq"], case["Hkv"], case["B"]
        keys = n + M - 1
        blocks = -(-keys // case["block"])
        seen = float((n * M + M * (M - 1) // 2).sum())
        table = 4 * float((-(-keys // case["page"])).sum())
        return {"bytes": float(keys.sum()) * Hkv * 2 * D + float(blocks.sum()) * Hkv * 8 + table + 4 * B
                + 2 * B * M * Hq * D * _size(case["dtype"]), "flops": seen * Hq * (4 * D + 4)}
    Hkv, T = case["Hkv"], int(n.sum())
    first = start // case["block"]
    blocks = float((-(-(start + n) // case["block"]) - first).sum())
    table = 4 * float((-(-(start + n) // case["page"]) - start // case["page"]).sum()) + 8 * case["B"]
    if case["op"] == "read":
        return {"bytes": T * Hkv * 2 * D * (1 + _size(case["out"])) + blocks * Hkv * 8 + table,
                "flops": float(T * Hkv * 2 * D)}
    back = float((start + n - first * case["block"]).sum())
    e, Hq = _size(case["dtype"]), case["Hq"]
    # rows and queries read, codes and queries written; the touched blocks read
    # back as float32; the angles of each position
    return {"bytes": T * D * (2 * Hkv * (e + 1) + Hq * 2 * e) + back * Hkv * 2 * D * 5.0 + blocks * Hkv * 24
            + T * case["rot"] * 4 + table,
            "flops": T * (3.0 * (Hq + Hkv) * case["rot"] + 4.0 * 2 * Hkv * D) + back * Hkv * 2 * D}


# ------------------------------------------------------------------ exact
# (written apart from the plain forms: host loops over sequences and blocks; where
# the operator is defined by float32 roundings, as the codes are, numpy makes them)

def _np(x):
    return x.float().cpu().numpy()


def _rotate64(x, angles, interleaved):
    h = angles.shape[1]
    c, s = angles[:, None, :, 0].astype(np.float64), angles[:, None, :, 1].astype(np.float64)
    y = x.astype(np.float64)
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    u, w = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = u * c - w * s, w * c + u * s
    return y


def _exact_rope(case, seed):
    s = _prepare_rope(case, seed)
    angles = s["table"][s["positions"].long()].cpu().numpy()
    return torch.from_numpy(_rotate64(_np(s["x"]), angles, case["interleaved"]))


def _e4m3(u):
    a = np.abs(u.astype(np.float64))
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(a, 1e-30))), -6) - 3)
    return np.sign(u) * np.minimum(np.rint(a / step) * step, 448.0)


def _exact_write(case, seed):
    s = _prepare_write(case, seed)
    int8, R, page = case["code"] == "int8", case["block"], case["page"]
    top = np.float32(127 if int8 else 448)
    quant = (lambda u: np.clip(np.rint(u), -127, 127)) if int8 else _e4m3
    table, cu, start = (s[n].cpu().numpy().astype(np.int64) for n in ("table", "cu", "start"))
    cache = {n: _np(s[n]).astype(np.float64) for n in ("k", "v")}
    scale = {n: s[n].cpu().numpy().copy() for n in ("ks", "vs")}
    angles = s["rope"].cpu().numpy()
    where = np.concatenate([np.arange(st, st + m) for st, m in zip(start, np.diff(cu))])
    # the keys' rotation as the operator defines it, each float32 operation rounded
    h = angles.shape[1]
    c, sn = angles[where][:, None, :, 0], angles[where][:, None, :, 1]
    k = _np(s["k_new"]).copy()
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if case["interleaved"] else (slice(0, h), slice(h, 2 * h))
    u, w = k[..., a].copy(), k[..., b].copy()
    k[..., a], k[..., b] = u * c - w * sn, w * c + u * sn
    rows = {"k": k, "v": _np(s["v_new"])}
    back = {"k": [], "v": []}
    for i in range(case["B"]):
        n, p0 = int(cu[i + 1] - cu[i]), int(start[i])
        for blk in range(p0 // R, -(-(p0 + n) // R)):
            at = int(table[i, blk * R // page]) * page + blk * R % page
            lo, hi = max(p0, blk * R), min(p0 + n, blk * R + R)
            for name in ("k", "v"):
                x = rows[name][cu[i] + lo - p0:cu[i] + hi - p0].transpose(1, 0, 2)
                new = (np.abs(x).max((1, 2)) / top).astype(np.float32)
                if lo > blk * R:
                    was = scale[name + "s"][:, at // R]
                    new = np.maximum(new, was)
                    grown = new > was
                    f = np.where(grown, was / np.where(grown, new, 1), 1).astype(np.float32)
                    kept = cache[name][:, at:at + lo - blk * R]
                    again = quant((kept.astype(np.float32) * f[:, None, None]).astype(np.float32))
                    cache[name][:, at:at + lo - blk * R] = np.where(grown[:, None, None], again, kept)
                scale[name + "s"][:, at // R] = new
                d = np.where(new > 0, new, 1)[:, None, None]
                cache[name][:, at + lo - blk * R:at + hi - blk * R] = \
                    np.where(new[:, None, None] > 0, quant((x / d).astype(np.float32)), 0)
                value = cache[name][:, at:at + hi - blk * R] * new.astype(np.float64)[:, None, None]
                back[name].append(value.transpose(1, 0, 2))
    out = {"q": torch.from_numpy(_rotate64(_np(s["q"]), angles[where], case["interleaved"]))}
    for name in ("k", "v"):
        out[name] = torch.from_numpy(np.concatenate(back[name]))
        out[name + "s"] = torch.from_numpy(scale[name + "s"].astype(np.float64))
    return out


def _exact_read(case, seed):
    s = _prepare_read(case, seed)
    table, cu, start = (s[n].cpu().numpy().astype(np.int64) for n in ("table", "cu", "start"))
    out = {}
    for name in ("k", "v"):
        value = s[name].float().double()
        value = value.view(case["Hkv"], -1, case["block"], D) * s[name + "s"].double()[:, :, None, None]
        value = value.view(case["Hkv"], -1, D).transpose(0, 1)
        rows = []
        for i in range(case["B"]):
            t = np.arange(start[i], start[i] + cu[i + 1] - cu[i])
            rows.append(table[i, t // case["page"]] * case["page"] + t % case["page"])
        out[name] = value[torch.from_numpy(np.concatenate(rows)).to(DEV)]
    return out


def _exact_attend(case, seed):
    s = _prepare_attend(case, seed)
    B, M, Hq, Hkv, page = (case[n] for n in ("B", "M", "Hq", "Hkv", "page"))
    g, ctx = Hq // Hkv, s["ctx"].cpu().numpy()
    if float((ctx.astype(np.float64) + M).sum()) * M * Hq * 4 * D > 6e12:
        return None
    out = torch.empty((B, M, Hq, D), dtype=torch.float64, device=DEV)
    for b in range(B):
        n = int(ctx[b]) + M - 1
        pages = s["table"][b, :(n + page - 1) // page].long()
        rows = (pages[:, None] * page + torch.arange(page, device=DEV)[None]).view(-1)[:n]
        for h in range(Hkv):
            key, value = (s[x][h].view(torch.uint8)[rows].view(s[x].dtype).double()
                          * s[x + "s"][h][rows // case["block"]].double()[:, None] for x in ("k", "v"))
            score = torch.einsum("mgd,td->mgt", s["q"][b, :, h * g:h * g + g].double(), key) / math.sqrt(D)
            for j in range(M):
                score[j, :, int(ctx[b]) + j:] = -math.inf
            out[b, :, h * g:h * g + g] = torch.softmax(score, -1) @ value
    return out


def exact(case, seed):
    return {"rope": _exact_rope, "write": _exact_write, "read": _exact_read,
            "attend": _exact_attend}[case["op"]](case, seed)
