"""Cases of the operators around the paged cache: attention with a window and sinks, the
norm + rotation + append pass, and the page operations (extend, fork, free, compact, copy).

`run` computes them in plain torch operations in 32 bits, or, when `own` is set, through
the library's entry points. Page tables, positions and weights are what a serving program
holds before each call.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_BYTES = {"bf16": 2, "e4m3": 1, "e5m2": 1}
_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
_EPS = 1e-6


# ---------------------------------------------------------------------------- cases
def _attend_case(kind, batch, kv, q, heads, d, page, window, sinks, kv_type="bf16"):
    return {"op": "attend", "kind": kind, "batch": batch, "kv_lo": kv[0], "kv_hi": kv[1],
            "q_lo": q[0], "q_hi": q[1], "qo_heads": heads[0], "kv_heads": heads[1], "d": d, "page": page,
            "window": window, "sinks": sinks, "kv_type": kv_type}


def _append_case(mode, tokens, pad, heads, d, rotary, interleaved, page, kv_type="bf16"):
    return {"op": "append", "mode": mode, "tokens": tokens, "pad": pad, "qo_heads": heads[0],
            "kv_heads": heads[1], "d": d, "rotary": rotary, "interleaved": interleaved, "page": page,
            "kv_type": kv_type}


def _pages_case(op, rows, calls, len_lo, len_hi, pages, page, heads, d):
    return {"op": op, "rows": rows, "calls": calls, "len_lo": len_lo, "len_hi": len_hi,
            "pages": pages, "page": page, "kv_heads": heads, "d": d}


def listed():
    return [
        # one conversation being answered: a single row, where latency counts
        {"name": "decode_one"} | _attend_case("decode", 1, (777, 777), (1, 1), (32, 8), 128, 16, 127, 4),
        # a decode batch of mixed lengths under a short window
        {"name": "decode_batch"} | _attend_case("decode", 64, (256, 4096), (1, 1), (32, 8), 128, 16, 1023, 4),
        # many long conversations over an 8-bit cache
        {"name": "decode_long_e4m3"} | _attend_case("decode", 256, (6000, 8192), (1, 1), (64, 8), 128, 16, 4095, 128, "e4m3"),
        # chunks of new tokens behind cached prefixes
        {"name": "extend"} | _attend_case("prefill", 8, (2048, 6000), (128, 2048), (32, 8), 128, 16, 2047, 4),
        # prompts of a small sliding-window model, token-granular pages
        {"name": "prefill_d256_page_1"} | _attend_case("prefill", 8, (1500, 1500), (1500, 1500), (4, 1), 256, 1, 511, 5),
        # one decode step of a batch, captured with a few padding rows behind it
        {"name": "append_decode"} | _append_case("scatter", 61, 3, (32, 8), 128, 128, False, 16),
        # prompt tokens of several requests
        {"name": "append_prompt"} | _append_case("runs", 16384, 0, (32, 8), 128, 128, False, 16),
        # an 8-bit cache, partly rotated heads, rows in no round number
        {"name": "append_prompt_e4m3"} | _append_case("runs", 8191, 17, (8, 4), 256, 64, True, 5, "e4m3"),
        # a beam step: few rows split, their last pages copied
        {"name": "fork_beams"} | _pages_case("fork", 64, 16, 100, 2000, 16384, 16, 8, 128),
        # a shared prompt sampled many times
        {"name": "fork_prompt"} | _pages_case("fork", 64, 512, 500, 4000, 16384, 16, 8, 128),
        # a pool at half load packed together
        {"name": "compact"} | _pages_case("compact", 256, 0, 100, 2000, 32768, 16, 8, 128),
        # a step of a large server: rows that ended are freed and their places filled again
        {"name": "recycle"} | _pages_case("recycle", 1024, 256, 10, 4000, 300000, 16, 0, 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "fork", "compact", "recycle"])
    page = rng.choice([1, 3, 8, 16, 16, 32, 64, 128])
    d = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    if op == "attend":
        kind = rng.choice(["decode", "decode", "prefill", "ragged"])
        kv_type = "bf16" if kind == "ragged" else rng.choice(["bf16", "bf16", "e4m3", "e5m2"])
        window, sinks = _log(rng, 1, 4095), _log(rng, 1, 200)
        if kind == "decode":
            hi = _log(rng, 20, 8192)
            return _attend_case(kind, _log(rng, 1, 200), (max(1, hi // rng.randint(1, 8)), hi), (1, 1),
                                (kv_heads * group, kv_heads), d, page, window, sinks, kv_type)
        hi = _log(rng, 20, 4000)
        q_hi = max(1, min(hi, _log(rng, 1, 1500)))
        return _attend_case(kind, _log(rng, 1, 6), (max(q_hi, hi // rng.randint(1, 4)), hi),
                            (max(1, q_hi // rng.randint(1, 4)), q_hi), (kv_heads * group, kv_heads), d, page,
                            window, sinks, kv_type)
    if op == "append":
        return _append_case(rng.choice(["scatter", "runs"]), _log(rng, 1, 12000), rng.choice([0, 0, 1, 9]),
                            (kv_heads * group, kv_heads), d, rng.choice([d, d, d // 2, 16]),
                            rng.random() < 0.4, page, rng.choice(["bf16", "bf16", "e4m3", "e5m2"]))
    rows = _log(rng, 4, 400)
    hi = _log(rng, 3, 1500)
    lo = max(1, hi // rng.randint(1, 20))
    need = rows * (-(-hi // page) + 1)
    calls = 0 if op == "compact" else _log(rng, 1, rows if op == "recycle" else 300)
    pages = int((need + calls) * rng.uniform(1.2, 3.0)) + 2
    if op == "recycle":
        return _pages_case(op, rows, calls, lo, hi, pages, page, 0, 0)
    d = min(d, 128)
    page_bytes = 2 * page * kv_heads * d
    while pages * page_bytes > (1 << 30):  # a drawn pool stays below the largest listed one
        if page > 1:
            page, pages = page // 2, pages
            page_bytes //= 2
            hi, lo = max(1, hi // 2), max(1, lo // 2)
        else:
            rows, pages = max(4, rows // 2), pages // 2
    need = rows * (-(-hi // page) + 1) + calls
    return _pages_case(op, rows, calls, lo, hi, max(pages, need + 2), page, kv_heads, d)


# ---------------------------------------------------------------------------- inputs
def _fixed(case):
    """The lengths of a case: the same for every seed, as `work` counts them."""
    return np.random.default_rng(abs(hash(tuple(v for k, v in sorted(case.items()) if isinstance(v, int)))) % (1 << 31))


def _attend_lens(case):
    rng = _fixed(case)
    kv = rng.integers(case["kv_lo"], case["kv_hi"] + 1, size=case["batch"])
    q = np.minimum(rng.integers(case["q_lo"], case["q_hi"] + 1, size=case["batch"]), kv)
    return kv.astype(np.int64), q.astype(np.int64)


def _page_lens(case):
    return _fixed(case).integers(case["len_lo"], case["len_hi"] + 1, size=case["rows"]).astype(np.int64)


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32), device="cuda")


def _i64(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int64), device="cuda")


def _offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def _prepare_attend(case, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    kv, ql = _attend_lens(case)
    B, P, d, hkv = case["batch"], case["page"], case["d"], case["kv_heads"]
    ragged = case["kind"] == "ragged"
    npg = kv if ragged else -(-kv // P)
    used = int(npg.sum())
    pool = used if ragged else int(used * 1.25) + 1
    pages = np.arange(used) if ragged else rng.permutation(pool)[:used]
    dtype = _TYPES[case["kv_type"]]
    shape = (pool, hkv, d) if ragged else (pool, P, hkv, d)
    kv_indptr, qo_indptr = _offsets(npg), _offsets(ql)
    last = kv - (npg - 1) * P
    s = {"case": case, "q": _randn(g, (int(ql.sum()), case["qo_heads"], d), torch.bfloat16),
         "k": _randn(g, shape, dtype), "v": _randn(g, shape, dtype), "kv_indices": _i32(pages),
         "kv_indptr": _i64(kv_indptr), "qo_indptr": _i64(qo_indptr), "kv_lens": _i64(kv), "q_lens": _i64(ql),
         "row_req": _i64(np.repeat(np.arange(B), ql)), "row_tok": _i64(np.concatenate([np.arange(n) for n in ql])),
         "max_kv": int(kv.max()), "max_q": int(ql.max()), "scale": d ** -0.5,
         "k_scale": 1.0 if case["kv_type"] == "bf16" else 0.75, "v_scale": 1.0 if case["kv_type"] == "bf16" else 1.5}
    if own:
        from paged_kv_sliding_gb300 import pkv
        kinds = {"decode": "decode", "prefill": "prefill", "ragged": "prefill_ragged"}
        s["plan"] = pkv.Plan(kind=kinds[case["kind"]], kv_indptr=kv_indptr, kv_indices=None if ragged else s["kv_indices"],
                             kv_last_page_len=None if ragged else last, num_qo_heads=case["qo_heads"],
                             num_kv_heads=hkv, head_dim=d, page_size=1 if ragged else P, num_pages=pool,
                             window_left=case["window"], num_sinks=case["sinks"], causal=True, sm_scale=s["scale"],
                             qo_indptr=None if case["kind"] == "decode" else qo_indptr, k_scale=s["k_scale"],
                             v_scale=s["v_scale"], kv_dtype=case["kv_type"])
    return s


_TABLE = 40000  # positions of the rotation table


def _prepare_append(case, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, pad, P, d = case["tokens"], case["pad"], case["page"], case["d"]
    hq, hkv, r = case["qo_heads"], case["kv_heads"], case["rotary"]
    if case["mode"] == "scatter":  # one token of each request, each in its own page
        pool = n + n // 4 + 2
        slots = rng.permutation(pool)[:n].astype(np.int64) * P + rng.integers(0, P, size=n)
        pos = rng.integers(0, _TABLE, size=n)
    else:  # runs of tokens that fill pages
        used = -(-n // P)
        pool = used + used // 8 + 2
        slots = rng.permutation(pool)[np.arange(n) // P].astype(np.int64) * P + np.arange(n) % P
        pos = (rng.integers(0, _TABLE) + np.arange(n)) % _TABLE
    slots = np.concatenate([slots, np.full(pad, -1)])
    pos = np.concatenate([pos, np.zeros(pad, dtype=np.int64)])
    angle = torch.arange(_TABLE, dtype=torch.float64, device="cuda")[:, None] * \
        (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r))[None]
    dtype = _TYPES[case["kv_type"]]
    cache = (pool, P, hkv, d)
    return {"case": case, "qkv": _randn(g, (n + pad, (hq + 2 * hkv) * d), torch.bfloat16) * 1.5,
            "slots": _i64(slots), "positions": _i32(pos),
            "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float(),
            "wq": _randn(g, (d,), torch.bfloat16) * 0.2, "wk": _randn(g, (d,), torch.bfloat16) * 0.2,
            "q_out": torch.full((n + pad, hq, d), 0.5, dtype=torch.bfloat16, device="cuda"),
            "k": torch.full(cache, 0.5, device="cuda").to(dtype), "v": torch.full(cache, -0.5, device="cuda").to(dtype),
            "k_scale": 1.0 if case["kv_type"] == "bf16" else 0.021, "v_scale": 1.0 if case["kv_type"] == "bf16" else 0.013}


def _prepare_pages(case, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, calls, P, pool = case["rows"], case["calls"], case["page"], case["pages"]
    lens = _page_lens(case)
    npg = -(-lens // P)
    total_rows = rows + (calls if case["op"] == "fork" else 0)
    cols = -(-case["len_hi"] // P) + 1
    used = int(npg.sum())
    ids = rng.permutation(pool)[:used].astype(np.int32)
    table = np.zeros((total_rows, cols), dtype=np.int32)
    table[:rows][np.arange(cols)[None] < npg[:, None]] = ids
    refs = np.zeros(pool, dtype=np.int32)
    refs[ids] = 1
    if case["op"] == "compact":  # a third of the rows share their first pages with the row before
        for i in range(2, rows, 3):
            k = int(min(lens[i], lens[i - 1]) // P)
            refs[table[i, :k]] -= 1
            table[i, :k] = table[i - 1, :k]
            refs[table[i, :k]] += 1
    s = {"case": case, "table": _i32(table), "lens": _i32(np.concatenate([lens, np.zeros(total_rows - rows)])),
         "refs": _i32(refs)}
    if case["op"] == "fork":
        s["parents"] = _i32(rng.integers(0, rows, size=calls))
        s["children"] = _i32(rows + rng.permutation(calls))
    elif case["op"] == "recycle":
        who = _fixed(case).permutation(rows)[:calls]
        s["rows"] = _i32(who)
        s["add"] = _i32(lens[who][::-1])
        s["total"] = int(lens[who].sum())
    if case["op"] == "compact":
        s["out_table"], s["out_refs"] = torch.zeros_like(s["table"]), torch.zeros_like(s["refs"])
        s["src"] = torch.full((pool // 2,), -1, dtype=torch.int32, device="cuda")
        s["dst"] = s["src"].clone()
    if case["op"] != "recycle":
        shape = (pool, P, case["kv_heads"], case["d"])
        s["k"], s["v"] = _randn(g, shape, torch.bfloat16), _randn(g, shape, torch.bfloat16)
    if own:
        from paged_kv_sliding_gb300 import pkv
        s["pool"] = pkv.PagePool(s["table"], s["lens"], s["refs"], page_size=P)
        if case["op"] == "compact":
            s["out_pool"] = pkv.PagePool(s["out_table"], torch.zeros_like(s["lens"]), s["out_refs"], page_size=P)
    return s


def prepare(case, seed):
    return {"attend": _prepare_attend, "append": _prepare_append}.get(case["op"], _prepare_pages)(case, seed)


# ---------------------------------------------------------------------------- plain forms
def _attend(s):
    c = s["case"]
    P, W, n_sinks = c["page"], c["window"], c["sinks"]
    hkv, grp, d, B = c["kv_heads"], c["qo_heads"] // c["kv_heads"], c["d"], c["batch"]
    kv_len = s["kv_lens"][:, None]
    if c["kind"] == "decode":  # the keys of the sinks, then of the window
        p = kv_len - 1
        a = torch.arange(n_sinks, device="cuda").expand(B, n_sinks)
        b = p - W + torch.arange(W + 1, device="cuda")
        j = torch.cat([a, b], 1)
        ok = torch.cat([(a < p - W) & (a < kv_len), b >= 0], 1)[:, None]
        n_q = 1
    else:
        n_q = s["max_q"]
        j = torch.arange(s["max_kv"], device="cuda").expand(B, -1)
        p = kv_len - s["q_lens"][:, None] + torch.arange(n_q, device="cuda")
        ok = (j < kv_len)[:, None] & (j[:, None] <= p[..., None]) & \
            ((j < n_sinks)[:, None] | (j[:, None] >= p[..., None] - W))
    jc = torch.minimum(j.clamp(min=0), kv_len - 1)
    if c["kind"] == "ragged":
        loc = s["kv_indptr"][:-1, None] + jc
    else:
        loc = s["kv_indices"][s["kv_indptr"][:-1, None] + jc // P].long() * P + jc % P
    k = s["k"].view(-1, hkv, d).view(torch.uint8 if s["k"].element_size() == 1 else s["k"].dtype)[loc].view(s["k"].dtype)
    v = s["v"].view(-1, hkv, d).view(torch.uint8 if s["v"].element_size() == 1 else s["v"].dtype)[loc].view(s["v"].dtype)
    k = k.float().permute(0, 2, 3, 1)  # [B, H_kv, d, keys]
    v = v.float().permute(0, 2, 1, 3)
    rows = (s["qo_indptr"][:-1, None] + torch.minimum(torch.arange(n_q, device="cuda")[None], s["q_lens"][:, None] - 1))
    q = s["q"][rows].float().view(B, n_q, hkv, grp, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, grp * n_q, d)
    x = torch.matmul(q, k).mul_(s["scale"] * s["k_scale"]).view(B, hkv, grp, n_q, -1)
    x.masked_fill_(~ok[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, hkv, grp * n_q, -1), v).view(B, hkv, grp, n_q, d) / l * s["v_scale"]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n_q, hkv * grp, d)
    lse = (m + l.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, n_q, hkv * grp)
    return {"out": o[s["row_req"], s["row_tok"]].to(torch.bfloat16), "lse": lse[s["row_req"], s["row_tok"]]}


def _norm_rotate(x, w, cos, sin, interleaved):
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * (w.float() + 1.0)
    h = cos.shape[-1]
    head, rest = x[..., : 2 * h], x[..., 2 * h:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = head[..., :h], head[..., h:]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([head, rest], -1)


def _store(cache, slots, x, scale, kv_type):
    flat = cache.view(-1, *cache.shape[2:])
    if kv_type == "bf16":
        flat[slots] = x.to(torch.bfloat16)
    else:
        x = (x / scale).clamp(-_MAX[kv_type], _MAX[kv_type]).to(_TYPES[kv_type])
        flat.view(torch.uint8)[slots] = x.view(torch.uint8)


def _append(s):
    c = s["case"]
    d, hq, hkv = c["d"], c["qo_heads"], c["kv_heads"]
    q, k, v = (x.view(-1, x.shape[1] // d, d).float() for x in s["qkv"].split([hq * d, hkv * d, hkv * d], 1))
    cs = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = cs.chunk(2, -1)
    rows = (s["slots"] >= 0).nonzero().squeeze(1)
    slots = s["slots"][rows]
    s["q_out"][rows] = _norm_rotate(q, s["wq"], cos, sin, c["interleaved"])[rows].to(torch.bfloat16)
    _store(s["k"], slots, _norm_rotate(k, s["wk"], cos, sin, c["interleaved"])[rows], s["k_scale"], c["kv_type"])
    _store(s["v"], slots, v[rows], s["v_scale"], c["kv_type"])


def _free(table, lens, refs, rows, P):
    used = torch.arange(table.shape[1], device="cuda")[None] < ((lens[rows] + P - 1) // P)[:, None]
    refs.scatter_add_(0, table[rows].long().flatten(), -used.int().flatten())
    lens[rows] = 0


def _lowest_free(refs):
    """free[r]: the r-th free page, ascending (one spare entry behind the last page)."""
    n = refs.shape[0]
    is_free = refs == 0
    rank = torch.where(is_free, is_free.cumsum(0) - 1, torch.full_like(refs, n, dtype=torch.int64))
    free = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    return free.scatter_(0, rank, torch.arange(n, dtype=torch.int32, device="cuda"))


def _fork(s):
    table, lens, refs, P = s["table"], s["lens"], s["refs"], s["case"]["page"]
    parents, children = s["parents"].long(), s["children"].long()
    _free(table, lens, refs, children, P)
    plen = lens[parents]
    full, part = (plen // P)[:, None], plen % P > 0
    new = _lowest_free(refs)[part.cumsum(0) - part.int()]
    src_row = table[parents]
    col = torch.arange(table.shape[1], device="cuda")[None]
    last = src_row.gather(1, full.long().clamp(max=table.shape[1] - 1)).squeeze(1)
    table[children] = torch.where(col < full, src_row, torch.where((col == full) & part[:, None], new[:, None], table[children]))
    refs.scatter_add_(0, src_row.long().flatten(), (col < full).int().flatten())
    refs.scatter_add_(0, new.long(), part.int())
    lens[children] = plen
    src, dst = torch.where(part, last, -1), torch.where(part, new, -1)
    a, b = src[part].long(), dst[part].long()
    s["k"][b] = s["k"][a]
    s["v"][b] = s["v"][a]
    return src, dst


def _compact(s):
    table, refs, P = s["table"], s["refs"], s["case"]["page"]
    n = refs.shape[0]
    ids = torch.arange(n, device="cuda")
    live = refs > 0
    n_live = live.sum()
    src, dst = ids[live & (ids >= n_live)], ids[~live & (ids < n_live)]
    new_id = ids.clone()
    new_id[src] = dst
    used = torch.arange(table.shape[1], device="cuda")[None] < ((s["lens"] + P - 1) // P)[:, None]
    s["out_table"].copy_(torch.where(used, new_id[table.long()].int(), s["out_table"]))
    s["out_refs"].copy_(refs)
    s["out_refs"][dst] = refs[src]
    s["out_refs"][src] = 0
    s["src"][: src.shape[0]] = src.int()
    s["dst"][: src.shape[0]] = dst.int()
    s["k"][dst] = s["k"][src]
    s["v"][dst] = s["v"][src]
    return torch.full((1,), src.shape[0], dtype=torch.int32, device="cuda")


def _recycle(s):
    table, lens, refs, P = s["table"], s["lens"], s["refs"], s["case"]["page"]
    rows, add = s["rows"].long(), s["add"].long()
    _free(table, lens, refs, rows, P)
    need = (add + P - 1) // P
    first = need.cumsum(0) - need
    col = torch.arange(table.shape[1], device="cuda")[None]
    mine = col < need[:, None]
    new = _lowest_free(refs)[torch.where(mine, first[:, None] + col, refs.shape[0])]
    table[rows] = torch.where(mine, new, table[rows])
    refs.scatter_add_(0, new.long().flatten(), mine.int().flatten())
    lens[rows] = s["add"]
    req = torch.repeat_interleave(torch.arange(rows.shape[0], device="cuda"), add, output_size=s["total"])
    tok = torch.arange(s["total"], device="cuda") - (add.cumsum(0) - add)[req]
    return table[rows[req], tok // P].long() * P + tok % P


# ---------------------------------------------------------------------------- the library's calls
def _run_own(s):
    from paged_kv_sliding_gb300 import pkv
    c = s["case"]
    if c["op"] == "attend":
        out, lse = s["plan"].run(s["q"], s["k"], s["v"], return_lse=True)
        return {"out": out, "lse": lse}
    if c["op"] == "append":
        d, hq, hkv = c["d"], c["qo_heads"], c["kv_heads"]
        q, k, v = (x.view(-1, x.shape[1] // d, d) for x in s["qkv"].split([hq * d, hkv * d, hkv * d], 1))
        pkv.norm_rope_append(q, k, v, positions=s["positions"], cos_sin=s["cos_sin"], slots=s["slots"], k_cache=s["k"],
                             v_cache=s["v"], q_weight=s["wq"], k_weight=s["wk"], eps=_EPS, weight_offset=1.0,
                             interleaved=c["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"], q_out=s["q_out"])
        return _appended(s)
    if c["op"] == "fork":
        s["pool"].free(s["children"])
        src, dst = s["pool"].fork(s["parents"], s["children"])
        pkv.copy_pages(s["k"], s["v"], src, dst)
        return _pool(s) | {"src": src, "dst": dst, "k": s["k"], "v": s["v"]}
    if c["op"] == "compact":
        src, dst, count = s["pool"].compact(out=s["out_pool"], src=s["src"], dst=s["dst"])
        pkv.copy_pages(s["k"], s["v"], src, dst, count=count)
        return {"table": s["out_table"], "refs": s["out_refs"], "src": src, "dst": dst, "count": count, "k": s["k"], "v": s["v"]}
    s["pool"].free(s["rows"])
    slots = s["pool"].extend(s["rows"], s["add"], total=s["total"])
    return _pool(s) | {"slots": slots}


def _pool(s):
    return {"table": s["table"], "lens": s["lens"], "refs": s["refs"]}


def _appended(s):
    # an 8-bit cache is handed back as the values it holds
    k, v = (x if s["case"]["kv_type"] == "bf16" else x.to(torch.bfloat16) for x in (s["k"], s["v"]))
    return {"q": s["q_out"], "k": k, "v": v}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "attend":
        return _attend(state)
    if op == "append":
        _append(state)
        return _appended(state)
    if op == "fork":
        src, dst = _fork(state)
        return _pool(state) | {"src": src, "dst": dst, "k": state["k"], "v": state["v"]}
    if op == "compact":
        count = _compact(state)
        return {"table": state["out_table"], "refs": state["out_refs"], "src": state["src"], "dst": state["dst"],
                "count": count, "k": state["k"], "v": state["v"]}
    slots = _recycle(state)
    return _pool(state) | {"slots": slots}


# ---------------------------------------------------------------------------- counts
def work(case):
    if case["op"] == "attend":
        kv, ql = _attend_lens(case)
        W, n_sinks, d = case["window"], case["sinks"], case["d"]
        pairs = keys = 0
        for n, m in zip(kv.tolist(), ql.tolist()):
            p = np.arange(n - m, n)
            lo = np.maximum(0, p - W)
            pairs += int((p - lo + 1 + np.minimum(n_sinks, lo)).sum())
            keys += n - int(lo[0]) + min(n_sinks, int(lo[0]))
        rows = int(ql.sum()) * case["qo_heads"]
        return {"bytes": keys * case["kv_heads"] * d * 2 * _BYTES[case["kv_type"]] + rows * (4 * d + 4),
                "flops": 4 * d * pairs * case["qo_heads"]}
    if case["op"] == "append":
        n, d, hq, hkv = case["tokens"], case["d"], case["qo_heads"], case["kv_heads"]
        per = (hq + 2 * hkv) * d * 2 + hq * d * 2 + 2 * hkv * d * _BYTES[case["kv_type"]] + 4 * case["rotary"] + 12
        return {"bytes": n * per, "flops": n * (hq + hkv) * 8 * d}
    P = case["page"]
    lens = _page_lens(case)
    entries = int((-(-lens // P)).sum())
    page_bytes = 2 * 2 * P * case["kv_heads"] * case["d"]
    if case["op"] == "fork":
        mean = entries / case["rows"]
        part = float((lens % P > 0).mean())
        return {"bytes": int(case["calls"] * (2 * part * page_bytes + 8 * mean) + 4 * case["pages"]), "flops": 0}
    if case["op"] == "compact":
        moved = entries * (1 - entries / case["pages"])  # live pages above the live count, for pages drawn at random
        return {"bytes": int(moved * 2 * page_bytes + 8 * case["pages"] + 8 * entries), "flops": 0}
    share = case["calls"] / case["rows"]
    return {"bytes": int(4 * case["pages"] + share * (entries * 16 + 8 * lens.sum())), "flops": 0}


# ---------------------------------------------------------------------------- in 64 bits
def _grid(x, kv_type):
    """x rounded to the nearest value of an 8-bit format (ties to even, largest finite value at most)."""
    mant, low = (3, -6) if kv_type == "e4m3" else (2, -14)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** (low - mant - 2)))).clamp(min=low)
    step = torch.exp2(e - mant)
    return (torch.round(x / step) * step).clamp(-_MAX[kv_type], _MAX[kv_type])


def _exact_attend(s):
    c = s["case"]
    P, W, d, hkv = c["page"], c["window"], c["d"], c["kv_heads"]
    grp = c["qo_heads"] // hkv
    kv, ql = _attend_lens(c)
    begin, page0, out, lse = 0, 0, [], []
    for n, m in zip(kv.tolist(), ql.tolist()):
        if c["kind"] == "ragged":
            k, v = s["k"][page0:page0 + n], s["v"][page0:page0 + n]
            page0 += n
        else:
            npg = -(-n // P)
            at = s["kv_indices"][page0:page0 + npg].long()
            k, v = (x.view(torch.uint8)[at].view(x.dtype).reshape(-1, hkv, d)[:n] if x.element_size() == 1
                    else x[at].reshape(-1, hkv, d)[:n] for x in (s["k"], s["v"]))
            page0 += npg
        q = s["q"][begin:begin + m].double()
        begin += m
        p = torch.arange(n - m, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")[None]
        hidden = (j > p) | ((j < p - W) & (j >= c["sinks"]))
        o = torch.empty(m, c["qo_heads"], d, dtype=torch.float64, device="cuda")
        z = torch.empty(m, c["qo_heads"], dtype=torch.float64, device="cuda")
        for h in range(c["qo_heads"]):
            x = q[:, h] @ k[:, h // grp].double().T * (s["scale"] * s["k_scale"])
            x = torch.where(hidden, -math.inf, x)
            z[:, h] = torch.logsumexp(x, 1)
            o[:, h] = torch.exp(x - z[:, h:h + 1]) @ v[:, h // grp].double() * s["v_scale"]
        out.append(o)
        lse.append(z)
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _exact_append(s):
    c = s["case"]
    n, d, hq, hkv, h = c["tokens"], c["d"], c["qo_heads"], c["kv_heads"], c["rotary"] // 2
    x = s["qkv"][:n].double().view(n, hq + 2 * hkv, d)
    table = s["cos_sin"].double()[s["positions"][:n].long()]
    turn = torch.complex(table[:, :h], table[:, h:])[:, None]

    def rotated(y, w):
        y = y / (y.pow(2).sum(-1, keepdim=True) / d + _EPS).sqrt() * (1.0 + w.double())
        y = y.clone()
        if c["interleaved"]:
            z = torch.view_as_complex(y[..., : 2 * h].reshape(n, -1, h, 2).contiguous()) * turn
            y[..., : 2 * h] = torch.view_as_real(z).reshape(n, -1, 2 * h)
        else:
            z = torch.complex(y[..., :h], y[..., h:2 * h]) * turn
            y[..., :h], y[..., h:2 * h] = z.real, z.imag
        return y

    q = s["q_out"].double().clone()
    q[:n] = rotated(x[:, :hq], s["wq"])
    out = {"q": q}
    for name, y, scale in (("k", rotated(x[:, hq:hq + hkv], s["wk"]), s["k_scale"]), ("v", x[:, hq + hkv:], s["v_scale"])):
        flat = s[name].to(torch.float64).view(-1, hkv, d).clone()
        flat[s["slots"][:n]] = y if c["kv_type"] == "bf16" else _grid(y / scale, c["kv_type"])
        out[name] = flat.view(s[name].shape)
    return out


def exact(case, seed):
    """The floating outputs from the definitions in 64 bits; the page operations give whole
    numbers and copies, which have no rounding to speak of."""
    if case["op"] == "attend":
        return _exact_attend(prepare(case, seed))
    if case["op"] == "append":
        return _exact_append(prepare(case, seed))
    return None
