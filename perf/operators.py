"""Measured cases of the paged-cache operators: what a serving loop does between and around
the group attention calls.

write    hs2_kv_write + hs2_kv_read: new rows (one token or a prompt's) into an FP4 / FP8 / bf16
         paged cache, quantised on the way, and the values they stand for read back.
attend   hs2_fa_chunk: causal attention of a ragged batch of query chunks (one token up to a
         prompt chunk per sequence) over a paged 4-bit, 8-bit or bf16 cache, with an optional
         sliding window and sink logits.
branch   hs2_pages_fork + hs2_pages_grow + hs2_pages_free: sequences forked into branches that
         share their full pages, room for a few tokens each, and the branches dropped again.
compact  hs2_pages_compact: the live pages of a fragmented pool moved to its front.

``own`` false: plain torch; true: the calls of ``top_hs2_fa_gb300.hs2``.
"""
import math

import torch

own = False

PAGE = 64
DEV = "cuda"
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # a chat turn's prompt chunk against its 32K history in a 4-bit cache
        dict(name="attend prompt chunk fp4", op="attend", dtype="fp4", batch=1, n_lo=2048, n_hi=2048, t_lo=32768,
             t_hi=32768, Hq=32, Hkv=4, d=128, w=0, sink=False),
        # four draft tokens of each of 64 requests verified against 16K-32K keys in 4 bits
        dict(name="attend drafts fp4", op="attend", dtype="fp4", batch=64, n_lo=4, n_hi=4, t_lo=16384, t_hi=32768,
             Hq=32, Hkv=4, d=128, w=0, sink=False),
        # single tokens of a few short requests: latency
        dict(name="attend tokens small fp4", op="attend", dtype="fp4", batch=4, n_lo=1, n_hi=1, t_lo=129, t_hi=1500,
             Hq=32, Hkv=4, d=128, w=0, sink=False),
        # continuous batching, multi-query heads: some requests bring one token, others a chunk
        dict(name="attend mixed fp8", op="attend", dtype="fp8", batch=12, n_lo=1, n_hi=700, t_lo=1000, t_hi=6000,
             Hq=32, Hkv=1, d=128, w=0, sink=False),
        # sliding-window layer with sinks over a ragged batch of prompt chunks, 64-wide heads
        dict(name="attend window bf16", op="attend", dtype="bf16", batch=8, n_lo=333, n_hi=1200, t_lo=1200, t_hi=4100,
             Hq=16, Hkv=2, d=64, w=128, sink=True),
        # a decode step's new rows, one per sequence
        dict(name="write tokens fp4", op="write", dtype="fp4", rows="bf16", batch=64, n_lo=1, n_hi=1, t_lo=16384,
             t_hi=32768, Hkv=4, d=128),
        # a whole prompt's bridged rows
        dict(name="write prompt fp4", op="write", dtype="fp4", rows="bf16", batch=1, n_lo=32768, n_hi=32768,
             t_lo=32768, t_hi=32768, Hkv=4, d=128),
        # ragged chunks of float32 rows into an 8-bit cache, page-unaligned on both sides
        dict(name="write ragged fp8", op="write", dtype="fp8", rows="f32", batch=24, n_lo=1, n_hi=900, t_lo=901,
             t_hi=5000, Hkv=2, d=64),
        # a few short requests branched once
        dict(name="branch small", op="branch", batch=4, children=8, t_lo=130, t_hi=1400, ahead=4, caches=1, Hkv=1,
             d=64),
        # a draft tree over 16 requests: four branches each, two caches on one table
        dict(name="branch drafts", op="branch", batch=16, children=64, t_lo=4096, t_hi=16384, ahead=70, caches=2,
             Hkv=4, d=128),
        # a small pool after most of its requests ended
        dict(name="compact small", op="compact", batch=12, t_lo=100, t_hi=1500, keep=3, caches=1, Hkv=1, d=128),
        # a serving pool after half of its requests ended
        dict(name="compact serving", op="compact", batch=64, t_lo=4096, t_hi=12288, keep=2, caches=1, Hkv=4, d=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "write", "write", "branch", "compact"))
    if op == "attend":
        d, hkv = rng.choice((64, 128)), rng.choice((1, 2, 4))
        g = rng.choice((1, 4, 8, 16)) if hkv > 1 else rng.choice((8, 16, 32))
        batch, n_hi = _log_int(rng, 1, 32), _log_int(rng, 1, 1500)
        n_lo = _log_int(rng, 1, n_hi)
        t_hi = n_hi + _log_int(rng, 1, 16000)
        # no more (query head, key) pairs, padded, than the largest listed case has
        while batch > 1 and batch * n_hi * hkv * g * t_hi > 1 << 31:
            batch //= 2
        n_hi = max(n_lo, min(n_hi, (1 << 31) // (batch * hkv * g * t_hi)))
        n_lo, t_hi = min(n_lo, n_hi), max(t_hi, n_hi)
        return dict(op=op, dtype=rng.choice(("fp4", "fp4", "fp8", "bf16")), batch=batch, n_lo=n_lo, n_hi=n_hi,
                    t_lo=rng.randint(n_hi, t_hi), t_hi=t_hi, Hq=hkv * g, Hkv=hkv, d=d,
                    w=rng.choice((0, 0, 128, _log_int(rng, 1, 2000))), sink=rng.random() < 0.4)
    if op == "write":
        d, hkv, batch, n_hi = rng.choice((64, 128)), rng.choice((1, 2, 4)), _log_int(rng, 1, 64), _log_int(rng, 1, 8000)
        n_hi = min(n_hi, 32768 // batch)
        return dict(op=op, dtype=rng.choice(("fp4", "fp4", "fp8")), rows=rng.choice(("bf16", "f32")), batch=batch,
                    n_lo=_log_int(rng, 1, n_hi), n_hi=n_hi, t_lo=n_hi, t_hi=n_hi + _log_int(rng, 1, 3000), Hkv=hkv,
                    d=d)
    if op == "branch":
        t_lo, batch = _log_int(rng, 1, 4000), _log_int(rng, 1, 16)
        return dict(op=op, batch=batch, children=_log_int(rng, 1, 64), t_lo=t_lo, t_hi=t_lo + _log_int(rng, 1, 4000),
                    ahead=_log_int(rng, 1, 200), caches=rng.choice((1, 2)), Hkv=rng.choice((1, 2, 4)),
                    d=rng.choice((64, 128)))
    t_lo = _log_int(rng, 64, 3000)
    return dict(op=op, batch=_log_int(rng, 2, 64), t_lo=t_lo, t_hi=t_lo + _log_int(rng, 1, 4000),
                keep=rng.choice((2, 3, 5)), caches=1, Hkv=rng.choice((1, 2, 4)), d=rng.choice((64, 128)))


def _lengths(lo, hi, batch, log=False):
    """`batch` lengths spread over [lo, hi], in a mixed order and mostly odd; both ends occur."""
    if batch == 1:
        return [hi]
    step = next(s for s in (7, 11, 13, 17) if batch % s)
    got = []
    for i in range(batch):
        u = ((i * step) % batch) / (batch - 1)
        got.append(int(round(lo * (hi / lo) ** u)) if log else int(round(lo + (hi - lo) * u)))
    return got


def _counts(c):
    """Tokens of each sequence in this call, and its keys with them."""
    n = _lengths(c["n_lo"], c["n_hi"], c["batch"], log=True)
    return n, [max(a, b) for a, b in zip(_lengths(c["t_lo"], c["t_hi"], c["batch"]), n)]


def _row_bytes(dtype, d):
    return {"bf16": 2 * d, "fp8": d, "fp4": d // 2 + d // 16}[dtype]


def work(c):
    if c["op"] == "attend":
        n, t = _counts(c)
        nbytes, pairs = 0, 0
        for ni, ti in zip(n, t):
            first = max(0, ti - ni - c["w"] + 1) if c["w"] else 0
            nbytes += 2 * (ti - first) * c["Hkv"] * _row_bytes(c["dtype"], c["d"]) + ni * c["Hq"] * (4 * c["d"] + 4)
            for p in (range(ti - ni, ti) if c["w"] else ()):
                pairs += min(c["w"], p + 1)
            pairs += 0 if c["w"] else ni * (ti - ni) + ni * (ni + 1) // 2
        return {"bytes": nbytes, "flops": 4 * pairs * c["Hq"] * c["d"]}
    if c["op"] == "write":
        values = 2 * sum(_counts(c)[0]) * c["Hkv"] * c["d"]
        stored = 2 * sum(_counts(c)[0]) * c["Hkv"] * _row_bytes(c["dtype"], c["d"])
        return {"bytes": values * (2 if c["rows"] == "bf16" else 4) + 2 * stored + values * 4, "flops": 4 * values}
    per_row = 2 * c["caches"] * c["Hkv"] * 2 * c["d"]
    t = _lengths(c["t_lo"], c["t_hi"], c["batch"])
    if c["op"] == "branch":
        kids = [t[s] for s in _sources(c)]
        entries = sum(-(-(k + c["ahead"]) // PAGE) for k in kids)
        return {"bytes": sum(2 * (k % PAGE) * per_row for k in kids) + 4 * 4 * entries, "flops": 0}
    live = [-(-v // PAGE) for i, v in enumerate(t) if i % c["keep"] == 0]
    pages = sum(-(-v // PAGE) for v in t)
    return {"bytes": 2 * (sum(live) * (pages - sum(live)) // pages) * PAGE * per_row + 4 * (2 * pages + 2 * sum(live)),
            "flops": 0}


def _sources(c):
    """The parent of each branch; some parents have several, the last slot none."""
    return [(i * 5 + i // 3) % c["batch"] for i in range(c["children"])]


# ---------------------------------------------------------------------------- inputs
def _e4m3_values(device):
    """The 127 finite non-negative E4M3 values, ascending by code, in 64 bits."""
    c = torch.arange(127, device=device)
    e, m = (c >> 3).double(), (c & 7).double()
    return torch.where(c < 8, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e - 7))


def _table(g, pages_of, num_pages, width):
    """A block table whose rows take pages of a random permutation of the pool, -1 behind."""
    order = torch.randperm(num_pages, generator=g, device=DEV).int()
    count = torch.tensor(pages_of, device=DEV)
    col = torch.arange(width, device=DEV)
    used = col[None, :] < count[:, None]
    rank = (torch.cumsum(used.flatten(), 0) - 1).clamp(min=0).view(used.shape)
    return torch.where(used, order[rank], -1).int().contiguous()


def _fill_fp4(x):
    """Codes and group scales near those of the rows `x` (float32 [pages, Hkv, 64, d]), slab scale 1/64."""
    g = x.view(*x.shape[:-1], -1, 16)
    sf = (g.abs().amax(-1) * (64 / 6)).to(torch.float8_e4m3fn)
    q = (g * 64 / sf.float().clamp(min=2.0 ** -9)[..., None]).view(x.shape)
    a = q.abs()
    code = sum((a > b).to(torch.uint8) for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)) + (q < 0).to(torch.uint8) * 8
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), sf.view(torch.uint8)


def _cache(g, dtype, num_pages, hkv, d, fill=True):
    """A cache's tensors: k, v and, where the type has them, k_scale, v_scale, k_sf, v_sf."""
    s = {}
    for side in ("k", "v"):
        shape = (num_pages, hkv, PAGE, d)
        if dtype == "bf16":
            s[side] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) if fill else \
                torch.zeros(shape, device=DEV, dtype=torch.bfloat16)
            continue
        # slab scales as a calibration gives them: near one value, no powers of two
        near = 1 / 16 if dtype == "fp8" else 1 / 64
        s[side + "_scale"] = near * (0.9 + 0.2 * torch.rand((num_pages, hkv), generator=g, device=DEV))
        if dtype == "fp8":
            s[side] = torch.zeros(shape, device=DEV, dtype=torch.uint8)
        else:
            s[side] = torch.zeros((num_pages, hkv, PAGE, d // 2), device=DEV, dtype=torch.uint8)
            s[side + "_sf"] = torch.zeros((num_pages, hkv, PAGE, d // 16), device=DEV, dtype=torch.uint8)
        for p in range(0, num_pages if fill else 0, 1024):
            x = torch.randn((min(1024, num_pages - p), *shape[1:]), generator=g, device=DEV)
            if dtype == "fp8":
                s[side][p:p + 1024] = (x * 16).to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                s[side][p:p + 1024], s[side + "_sf"][p:p + 1024] = _fill_fp4(x)
    return s


def _handle(s):
    """The framework's view of the cache (`own` only)."""
    from top_hs2_fa_gb300 import hs2

    return hs2.KV(k=s["k"], v=s["v"], block_table=s["table"], seq_len=s["seq_len"], k_scale=s.get("k_scale"),
                  v_scale=s.get("v_scale"), k_sf=s.get("k_sf"), v_sf=s.get("v_sf"))


def _starts(n):
    return torch.tensor([0] + n, device=DEV).cumsum(0).int()


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if c["op"] in ("attend", "write"):
        n, t = _counts(c)
        pages_of = [-(-v // PAGE) for v in t]
        s = _cache(g, c["dtype"], sum(pages_of) + 3, c["Hkv"], c["d"], fill=c["op"] == "attend")
        s.update(c=c, table=_table(g, pages_of, sum(pages_of) + 3, max(pages_of)), n_rows=sum(n), max_n=max(n),
                 max_t=max(t), seq_len=torch.tensor(t, device=DEV, dtype=torch.int32), row_start=_starts(n))
        if c["op"] == "attend":
            s["q"] = torch.randn((sum(n), c["Hq"], c["d"]), generator=g, device=DEV, dtype=torch.bfloat16)
            s["sink"] = torch.randn((c["Hq"],), generator=g, device=DEV) + 2 if c["sink"] else None
        else:
            # K and V rows as slices of a fused projection's output, a few channels much larger than the rest
            width = (2 * c["Hkv"] + 2) * c["d"]
            x = torch.randn((sum(n), width), generator=g, device=DEV)
            x *= 1 + 5 * (torch.rand((width,), generator=g, device=DEV) < 0.03)
            x = x.to(torch.bfloat16) if c["rows"] == "bf16" else x
            kd = c["Hkv"] * c["d"]
            s["k_rows"] = x[:, 2 * c["d"]:2 * c["d"] + kd].unflatten(1, (c["Hkv"], c["d"]))
            s["v_rows"] = x[:, 2 * c["d"] + kd:].unflatten(1, (c["Hkv"], c["d"]))
    else:
        t = _lengths(c["t_lo"], c["t_hi"], c["batch"])
        pages_of = [-(-v // PAGE) for v in t]
        width = max(pages_of) + 4
        num_pages = sum(pages_of)
        if c["op"] == "branch":
            num_pages += c["children"] * (c["ahead"] // PAGE + 2) + 5
        table = _table(g, pages_of, num_pages, width)
        s = dict(c=c, num_pages=num_pages, seq_len=torch.tensor(t, device=DEV, dtype=torch.int32),
                 caches=[_cache(g, "bf16", num_pages, c["Hkv"], c["d"]) for _ in range(c["caches"])])
        keep = torch.ones(c["batch"], device=DEV, dtype=torch.bool)
        if c["op"] == "compact":
            keep = torch.arange(c["batch"], device=DEV) % c["keep"] == 0
            s["seq_len"] = s["seq_len"][keep].contiguous()
            table = table[keep].contiguous()
        ref = torch.zeros(num_pages + 1, device=DEV, dtype=torch.int32)
        ref[torch.where(table >= 0, table, num_pages).flatten().long()] = 1
        ref = ref[:num_pages]
        free = torch.nonzero(ref == 0).flatten()
        free = free[torch.randperm(free.numel(), generator=g, device=DEV)]
        # the books of the pool in one buffer: table, references, free list, its length
        meta = torch.full((table.numel() + 2 * num_pages + 1,), -1, device=DEV, dtype=torch.int32)
        s["meta"], a, b = meta, table.numel(), table.numel() + num_pages
        s["table"], s["ref"], s["free_list"], s["n_free"] = meta[:a].view_as(table), meta[a:b], meta[b:-1], meta[-1:]
        s["table"].copy_(table)
        s["ref"].copy_(ref)
        s["free_list"][:free.numel()] = free.int()
        s["n_free"].fill_(free.numel())
        s["meta0"] = meta.clone()
        if c["op"] == "branch":
            s["src"] = torch.tensor(_sources(c), device=DEV, dtype=torch.int32)
            s["n_new"] = torch.full((c["children"],), c["ahead"], device=DEV, dtype=torch.int32)
            s["drop"] = torch.ones(c["children"], device=DEV, dtype=torch.int32)
    if own:
        from top_hs2_fa_gb300 import hs2

        if c["op"] in ("attend", "write"):
            s["kv"] = _handle(s)
            if c["op"] == "attend":
                s["ws"] = torch.empty(hs2.hs2_fa_chunk_workspace(s["n_rows"], c["Hq"], s["kv"], s["max_n"], s["max_t"],
                                                                 c["w"]), device=DEV, dtype=torch.uint8)
        else:
            s["kvs"] = [hs2.KV(k=x["k"], v=x["v"], block_table=s["table"], seq_len=s["seq_len"]) for x in s["caches"]]
            s["pages"] = hs2.Pages(ref=s["ref"], free_list=s["free_list"], n_free=s["n_free"])
            if c["op"] == "compact":
                s["ws"] = torch.empty(hs2.hs2_pages_compact_workspace(s["pages"]), device=DEV, dtype=torch.uint8)
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    op = s["c"]["op"]
    if op == "attend":
        return _attend_own(s) if own else _attend_plain(s)
    if op == "write":
        return _write_own(s) if own else _write_plain(s)
    if op == "branch":
        return _branch_own(s) if own else _branch_plain(s)
    return _compact_own(s) if own else _compact_plain(s)


def _attend_own(s):
    from top_hs2_fa_gb300 import hs2

    c = s["c"]
    o, lse = hs2.hs2_fa_chunk(s["q"], s["row_start"], s["kv"], c["d"] ** -0.5, s["max_n"], max_t=s["max_t"], w=c["w"],
                              sink=s["sink"], o_dtype=torch.bfloat16, workspace=s["ws"])
    return {"o": o, "lse": lse}


def _values(s, side, pages):
    """float32 values of the pages `pages` ([...] of page ids): [..., Hkv, 64, d]."""
    x, sf, scale = s[side][pages], s.get(side + "_sf"), s.get(side + "_scale")
    if scale is None:
        return x.float()
    if sf is None:
        return x.view(torch.float8_e4m3fn).float() * scale[pages][..., None, None]
    level = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=x.device)
    x = level[torch.stack((x & 15, x >> 4), -1).flatten(-2).int()]
    sf = sf[pages].view(torch.float8_e4m3fn).float()[..., None]
    return (x.unflatten(-1, (-1, 16)) * sf).flatten(-2) * scale[pages][..., None, None]


def _attend_plain(s):
    c, q = s["c"], s["q"]
    hkv, d, top = c["Hkv"], c["d"], s["max_n"]
    start, length = s["row_start"].long(), s["seq_len"].long()
    n = start[1:] - start[:-1]
    row = torch.arange(q.shape[0], device=q.device)
    b = torch.bucketize(row, start[1:], right=True)
    i = row - start[b]
    slot = (start[:-1, None] + torch.arange(top, device=q.device)).clamp(max=q.shape[0] - 1)
    x = q[slot].float().unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4)  # [B, Hkv, top, G, d]
    group = x.shape[3]
    pages = s["table"].clamp(min=0).long()
    k = _values(s, "k", pages).transpose(1, 2).flatten(2, 3)  # [B, Hkv, T, d]
    x = (x.flatten(2, 3) @ k.transpose(-1, -2)).mul_(d ** -0.5).unflatten(2, (top, group))
    del k
    at = (length - n)[:, None] + torch.arange(top, device=q.device)  # position of each query
    key = torch.arange(x.shape[-1], device=q.device)
    hidden = key > at[..., None]
    if c["w"]:
        hidden |= key <= at[..., None] - c["w"]
    x.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].view(1, hkv, 1, group, 1)
        m = torch.maximum(m, sink)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(sink - m)
    v = _values(s, "v", pages).transpose(1, 2).flatten(2, 3)
    # rows behind a table's end are page 0's: their weight is 0, and so is what they add
    o = (x.flatten(2, 3) @ v).unflatten(2, (top, group)) / total
    lse = (m + torch.log(total)).squeeze(-1)
    o, lse = o.permute(0, 2, 1, 3, 4).flatten(2, 3), lse.permute(0, 2, 1, 3).flatten(2, 3)
    return {"o": o[b, i].to(torch.bfloat16), "lse": lse[b, i]}


def _write_own(s):
    from top_hs2_fa_gb300 import hs2

    hs2.hs2_kv_write(s["kv"], s["k_rows"], s["v_rows"], s["row_start"])
    k, v = hs2.hs2_kv_read(s["kv"], s["row_start"], s["n_rows"])
    return {"k": k, "v": v}


def _nearest(a, borders):
    """How many of `borders` lie below `a`; on a border the even count of the two."""
    below, upto = torch.bucketize(a, borders, out_int32=True), torch.bucketize(a, borders, right=True, out_int32=True)
    return torch.where(below % 2 == 0, below, upto)


def _write_plain(s):
    c, out = s["c"], {}
    start = s["row_start"].long()
    row = torch.arange(s["n_rows"], device=start.device)
    b = torch.bucketize(row, start[1:], right=True)
    at = s["seq_len"].long()[b] - (start[1:] - start[:-1])[b] + row - start[b]
    page, line = s["table"][b, at // PAGE].long(), at % PAGE
    e4m3 = _e4m3_values(start.device)
    for side in ("k", "v"):
        x = s[side + "_rows"].double()  # ties and borders have to be seen exactly
        scale = s[side + "_scale"][page].double()[..., None]  # [n, Hkv, 1]
        sign = x.signbit()
        if c["dtype"] == "fp8":
            code = _nearest((x / scale).abs(), (e4m3[1:] + e4m3[:-1]) / 2)
            s[side][page, :, line] = torch.where(sign, code + 128, code).to(torch.uint8)
        else:
            amax = x.abs().unflatten(-1, (-1, 16)).amax(-1)
            sf = torch.bucketize(amax / (6 * scale), e4m3).clamp(max=126)  # the smallest that reaches
            unit = (e4m3[sf] * scale).repeat_interleave(16, -1)
            level = torch.tensor(_E2M1, device=x.device, dtype=torch.float64)
            code = _nearest(torch.where(unit > 0, (x / unit).abs(), 0.0), (level[1:] + level[:-1]) / 2)
            code = torch.where(sign, code + 8, code).to(torch.uint8)
            s[side][page, :, line] = code[..., 0::2] | (code[..., 1::2] << 4)
            s[side + "_sf"][page, :, line] = sf.to(torch.uint8)
        out[side] = _row_values(s, side, page, line)
    return out


def _row_values(s, side, page, line):
    x, sf, scale = s[side][page, :, line], s.get(side + "_sf"), s[side + "_scale"][page][..., None]
    if sf is None:
        return x.view(torch.float8_e4m3fn).float() * scale
    level = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=x.device)
    x = level[torch.stack((x & 15, x >> 4), -1).flatten(-2).int()]
    sf = sf[page, :, line].view(torch.float8_e4m3fn).float()[..., None]
    return (x.unflatten(-1, (-1, 16)) * sf).flatten(-2) * scale


def _pools(s):
    return [x[side] for x in s["caches"] for side in ("k", "v")]


def _branch_own(s):
    from top_hs2_fa_gb300 import hs2

    table, length = hs2.hs2_pages_fork(s["pages"], s["kvs"], s["src"])
    hs2.hs2_pages_grow(s["pages"], table, length, s["n_new"])
    hs2.hs2_pages_free(s["pages"], table, length, s["drop"])
    return {"table": table, "length": length, "ref": s["ref"], "n_free": s["n_free"], "free_list": s["free_list"],
            "pools": _pools(s)}


def _branch_plain(s):
    table, ref, free, n_free = s["table"], s["ref"], s["free_list"], s["n_free"]
    col = torch.arange(table.shape[1], device=table.device)
    src = s["src"].long()
    # fork: full pages shared, a page of its own for the rest
    length = s["seq_len"][src]
    full, rest = length // PAGE, length % PAGE
    child = torch.where(col < full[:, None], table[src], -1)
    ref.index_add_(0, child.clamp(min=0).flatten(), (child >= 0).flatten().int())
    takes = rest > 0
    rank = (torch.cumsum(takes, 0) - 1).clamp(min=0)
    new = free[(n_free - 1 - rank).clamp(min=0)].clamp(min=0)
    last = table[src].gather(1, full[:, None].long().clamp(max=table.shape[1] - 1))[:, 0]
    child = torch.where(takes[:, None] & (col == full[:, None]), new[:, None], child)
    ref.index_add_(0, new, takes.int())
    n_free -= takes.sum().int()
    line = torch.arange(PAGE, device=table.device)
    who, at = torch.nonzero(line < rest[:, None], as_tuple=True)
    to, of = new[who].long(), last[who].long()
    for pool in _pools(s):
        pool[to, :, at] = pool[of, :, at]
    # grow: pages for the tokens ahead
    have, length = (length + PAGE - 1) // PAGE, length + s["n_new"]
    need = (col >= have[:, None]) & (col < ((length + PAGE - 1) // PAGE)[:, None])
    rank = (torch.cumsum(need.flatten(), 0) - 1).clamp(min=0).view(need.shape)
    child = torch.where(need, free[(n_free - 1 - rank).clamp(min=0)], child)
    ref.index_add_(0, child.clamp(min=0).flatten(), need.flatten().int())
    n_free -= need.sum().int()
    # free: pages nobody refers to any more return in page order
    held = (col < ((length + PAGE - 1) // PAGE)[:, None]) & (s["drop"] != 0)[:, None]
    before = ref > 0
    ref.index_add_(0, child.clamp(min=0).flatten(), -held.flatten().int())
    gone = torch.nonzero(before & (ref == 0)).flatten()
    free[n_free + torch.arange(gone.numel(), device=free.device)] = gone.int()
    n_free += gone.numel()
    return {"table": child, "length": length, "ref": ref, "n_free": n_free, "free_list": free, "pools": _pools(s)}


def _compact_own(s):
    from top_hs2_fa_gb300 import hs2

    s["meta"].copy_(s["meta0"])  # the pass starts from the fragmented pool's books
    hs2.hs2_pages_compact(s["pages"], s["kvs"], workspace=s["ws"])
    return {"table": s["table"], "ref": s["ref"], "n_free": s["n_free"], "free_list": s["free_list"],
            "pools": _pools(s)}


def _compact_plain(s):
    s["meta"].copy_(s["meta0"])
    table, ref, free, n_free = s["table"], s["ref"], s["free_list"], s["n_free"]
    live, page = ref > 0, torch.arange(s["num_pages"], device=ref.device)
    count = live.sum()
    to, of = torch.nonzero(~live & (page < count)).flatten(), torch.nonzero(live & (page >= count)).flatten()
    for pool in _pools(s):
        pool[to] = pool[of]
    place = page.int()
    place[of] = to.int()
    col = torch.arange(table.shape[1], device=table.device)
    held = col < ((s["seq_len"] + PAGE - 1) // PAGE)[:, None]
    table.copy_(torch.where(held, place[table.clamp(min=0)], table))
    ref[to] = ref[of]
    ref.masked_fill_(page >= count, 0)
    n_free.copy_((s["num_pages"] - count).int().view(1))
    free.copy_(torch.where(page < n_free, s["num_pages"] - 1 - page, -1).int())
    return {"table": table, "ref": ref, "n_free": n_free, "free_list": free, "pools": _pools(s)}


# ---------------------------------------------------------------------------- 64 bits
def exact(c, seed):
    if c["op"] == "attend":
        return _attend_exact(prepare(c, seed))
    if c["op"] == "write":
        return _write_exact(prepare(c, seed))
    return None  # whole numbers and copies


def _byte_value(code, bias, man):
    """Value of float codes with `man` mantissa bits and exponent bias `bias` (no sign), in 64 bits."""
    exp, frac = code >> man, (code & ((1 << man) - 1)).double() / (1 << man)
    return torch.where(exp > 0, torch.ldexp(1 + frac, exp - bias), torch.ldexp(frac, torch.full_like(exp, 1 - bias)))


def _sequence64(s, side, pages):
    """All rows of the pages of one sequence, one head at a time: [Hkv, T, d] in 64 bits."""
    raw, c = s[side][pages].transpose(0, 1).flatten(1, 2), s["c"]
    if c["dtype"] == "bf16":
        return raw.double()
    slab = s[side + "_scale"][pages].double().T.repeat_interleave(PAGE, 1)[..., None]
    raw = raw.int()
    if c["dtype"] == "fp8":
        return _byte_value(raw & 127, 7, 3) * (1 - 2 * (raw >> 7)) * slab
    group = _byte_value(s[side + "_sf"][pages].transpose(0, 1).flatten(1, 2).int(), 7, 3)
    codes = torch.empty((*raw.shape[:-1], c["d"]), device=raw.device, dtype=torch.int32)
    codes[..., 0::2], codes[..., 1::2] = raw % 16, raw // 16
    return _byte_value(codes & 7, 1, 1) * (1 - 2 * (codes >> 3)) * group.repeat_interleave(16, -1) * slab


def _attend_exact(s):
    c = s["c"]
    start, length = s["row_start"].tolist(), s["seq_len"].tolist()
    group = c["Hq"] // c["Hkv"]
    o = torch.empty(s["q"].shape, device=DEV, dtype=torch.float64)
    lse = torch.empty(s["q"].shape[:2], device=DEV, dtype=torch.float64)
    for b in range(c["batch"]):
        t, r0, r1 = length[b], start[b], start[b + 1]
        pages = s["table"][b, :-(-t // PAGE)].long()
        k, v = _sequence64(s, "k", pages)[:, :t], _sequence64(s, "v", pages)[:, :t]
        pos = torch.arange(t - (r1 - r0), t, device=DEV)[:, None]
        key = torch.arange(t, device=DEV)[None, :]
        seen = (key <= pos) & (key > pos - (c["w"] or t + 1))
        for h in range(c["Hq"]):
            x = s["q"][r0:r1, h].double() @ k[h // group].T / math.sqrt(c["d"])
            x = torch.where(seen, x, -math.inf)
            if s["sink"] is not None:
                x = torch.cat((x, s["sink"][h].double().expand(r1 - r0, 1)), 1)
            z = torch.logsumexp(x, 1)
            o[r0:r1, h] = torch.exp(x[:, :t] - z[:, None]) @ v[h // group]
            lse[r0:r1, h] = z
    return {"o": o, "lse": lse}


def _write_exact(s):
    c, got = s["c"], {}
    start, length = s["row_start"].tolist(), s["seq_len"].tolist()
    pages = [s["table"][b, torch.arange(length[b] - (start[b + 1] - start[b]), length[b], device=DEV) // PAGE]
             for b in range(c["batch"])]
    page = torch.cat(pages).long()
    mag8 = _byte_value(torch.arange(127, device=DEV), 7, 3)
    mag4 = _byte_value(torch.arange(8, device=DEV), 1, 1)

    def closest(a, mags):
        # the nearest magnitude: of the largest not above and the smallest not below, an even code on a tie
        hi = torch.searchsorted(mags, a).clamp(max=mags.numel() - 1)
        lo = torch.where(mags[hi] > a, hi - 1, hi).clamp(min=0)
        up, down = mags[hi] - a, a - mags[lo]
        return mags[torch.where(up < down, hi, torch.where(down < up, lo, torch.where(lo % 2 == 0, lo, hi)))]

    for side in ("k", "v"):
        x, slab = s[side + "_rows"].double(), s[side + "_scale"][page].double()[..., None]
        sign = 1 - 2 * x.signbit().double()
        if c["dtype"] == "fp8":
            got[side] = sign * closest(x.abs() / slab, mag8) * slab
        else:
            a = x.abs().unflatten(-1, (-1, 16))
            top = a.amax(-1) / slab
            unit = mag8[torch.searchsorted(6 * mag8, top).clamp(max=126)]
            unit = (unit * slab)[..., None]
            got[side] = sign * (closest(torch.where(unit > 0, a / unit, 0.0), mag4) * unit).flatten(-2)
    return got
