"""Measured cases of the latent-attention operators and of the appends that rotate by position.

rotate   hs2_kv_write_rot + hs2_kv_read: new K, V rows into a paged cache and the queries beside them,
         K and queries rotated by their positions on the way; the values stored are read back.
append   hs2_latent_write + hs2_latent_read: new latent rows with their rotated key part into a paged
         latent cache, the queries' rotated part into its place beside the latent part.
absorbed hs2_latent_chunk: causal attention of a ragged batch over a paged latent cache, queries and
         outputs in the latent space (single tokens, drafts, chunks).
expanded hs2_latent_prefill: causal attention of prompts (or chunks with a history) over keys and
         values expanded from the latents, the rotated key part shared by the heads.

``own`` false: plain torch; true: the calls of ``top_hs2_fa_gb300.hs2``.
"""
import math

import torch

own = False

PAGE = 64
DEV = "cuda"
DR = 64  # rotated channels of a latent row
_SCALE = 192 ** -0.5  # of the expanded heads, whichever form runs


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's rows, one per sequence
        dict(name="rotate tokens bf16", op="rotate", dtype="bf16", rows="bf16", style="halves", rot=128, batch=64,
             n_lo=1, n_hi=1, t_lo=16384, t_hi=32768, Hq=32, Hkv=4, d=128),
        # a whole prompt into an 8-bit cache
        dict(name="rotate prompt fp8", op="rotate", dtype="fp8", rows="bf16", style="halves", rot=128, batch=1,
             n_lo=32768, n_hi=32768, t_lo=32768, t_hi=32768, Hq=32, Hkv=4, d=128),
        # ragged chunks of float32 rows, a part of the channels rotated, as neighbours
        dict(name="rotate ragged bf16", op="rotate", dtype="bf16", rows="f32", style="pairs", rot=32, batch=24, n_lo=1,
             n_hi=900, t_lo=901, t_hi=5000, Hq=16, Hkv=2, d=64),
        # a decode step's latent rows
        dict(name="append tokens", op="append", style="pairs", batch=64, n_lo=1, n_hi=1, t_lo=16384, t_hi=32768,
             Hq=128, dc=512),
        # ragged prompts' latent rows
        dict(name="append prompts", op="append", style="pairs", batch=8, n_lo=777, n_hi=8000, t_lo=777, t_hi=9000,
             Hq=32, dc=512),
        # single tokens of a few short requests: latency
        dict(name="absorbed tokens small", op="absorbed", batch=4, n_lo=1, n_hi=1, t_lo=129, t_hi=1500, Hq=16, dc=512),
        # a decode step of 64 long requests, the heads spread over several devices
        dict(name="absorbed tokens", op="absorbed", batch=64, n_lo=1, n_hi=1, t_lo=16384, t_hi=32768, Hq=16, dc=512),
        # a decode step with all the heads on one device
        dict(name="absorbed tokens all heads", op="absorbed", batch=32, n_lo=1, n_hi=1, t_lo=4096, t_hi=16384, Hq=128,
             dc=512),
        # continuous batching: some requests bring one token, others drafts or a short chunk
        dict(name="absorbed mixed", op="absorbed", batch=12, n_lo=1, n_hi=200, t_lo=1000, t_hi=6000, Hq=32, dc=512),
        # a few short prompts: latency
        dict(name="expanded small", op="expanded", batch=3, n_lo=17, n_hi=129, t_lo=17, t_hi=200, Hq=16),
        # a long prompt
        dict(name="expanded prompt", op="expanded", batch=1, n_lo=16384, n_hi=16384, t_lo=16384, t_hi=16384, Hq=16),
        # ragged chunks of prompts against their histories
        dict(name="expanded chunks", op="expanded", batch=8, n_lo=333, n_hi=1200, t_lo=1200, t_hi=6100, Hq=32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotate", "append", "absorbed", "absorbed", "absorbed", "expanded", "expanded"))
    if op == "rotate":
        d, hkv, batch, n_hi = rng.choice((64, 128)), rng.choice((1, 2, 4)), _log_int(rng, 1, 64), _log_int(rng, 1, 8000)
        n_hi = min(n_hi, 32768 // batch)
        return dict(op=op, dtype=rng.choice(("bf16", "fp8")), rows=rng.choice(("bf16", "f32")),
                    style=rng.choice(("halves", "pairs")), rot=rng.choice((32, 64, d)), batch=batch,
                    n_lo=_log_int(rng, 1, n_hi), n_hi=n_hi, t_lo=n_hi, t_hi=n_hi + _log_int(rng, 1, 3000),
                    Hq=hkv * rng.choice((1, 4, 8)), Hkv=hkv, d=d)
    if op == "append":
        batch, n_hi = _log_int(rng, 1, 64), _log_int(rng, 1, 8000)
        n_hi = min(n_hi, 32768 // batch)
        return dict(op=op, style=rng.choice(("halves", "pairs")), batch=batch, n_lo=_log_int(rng, 1, n_hi), n_hi=n_hi,
                    t_lo=n_hi, t_hi=n_hi + _log_int(rng, 1, 3000), Hq=rng.choice((8, 16, 32)),
                    dc=rng.choice((256, 512)))
    batch = _log_int(rng, 1, 32)
    if op == "absorbed":
        hq, n_hi, most = rng.choice((1, 8, 16, 32, 64, 128)), _log_int(rng, 1, 300), 1 << 27
        t_hi = n_hi + _log_int(rng, 1, 30000)
    else:
        hq, n_hi, most = rng.choice((8, 16, 32)), _log_int(rng, 1, 4000), 1 << 31
        t_hi = n_hi + rng.choice((0, _log_int(rng, 1, 8000)))
    n_lo = _log_int(rng, 1, n_hi)
    # no more (query head, key) pairs, padded, than the largest listed case has
    while batch > 1 and batch * n_hi * hq * t_hi > most:
        batch //= 2
    n_hi = max(1, min(n_hi, most // (batch * hq * t_hi)))
    c = dict(op=op, batch=batch, n_lo=min(n_lo, n_hi), n_hi=n_hi, t_lo=rng.randint(n_hi, t_hi), t_hi=t_hi, Hq=hq)
    return dict(c, dc=rng.choice((512, 512, 256))) if op == "absorbed" else c


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


def work(c):
    n, t = _counts(c)
    rows = sum(n)
    if c["op"] == "rotate":
        size, stored = (2 if c["rows"] == "bf16" else 4), (2 if c["dtype"] == "bf16" else 1)
        kv = 2 * c["Hkv"] * c["d"]
        per_row = kv * (size + 2 * stored + 2) + c["Hq"] * c["d"] * (size + 2) + 4 * c["rot"]
        return {"bytes": rows * per_row, "flops": 3 * rows * (c["Hkv"] + c["Hq"]) * c["rot"]}
    if c["op"] == "append":
        return {"bytes": rows * (8 * (c["dc"] + DR) + 4 * c["Hq"] * DR + 4 * DR), "flops": 3 * rows * (1 + c["Hq"]) * DR}
    pairs = sum(ni * (ti - ni) + ni * (ni + 1) // 2 for ni, ti in zip(n, t)) * c["Hq"]
    if c["op"] == "absorbed":
        d = c["dc"] + DR
        return {"bytes": 2 * sum(t) * d + rows * c["Hq"] * (2 * d + 2 * c["dc"] + 4),
                "flops": 2 * pairs * (d + c["dc"])}
    return {"bytes": sum(t) * 2 * (c["Hq"] * 256 + DR) + rows * c["Hq"] * (2 * 192 + 2 * 128 + 4),
            "flops": 2 * pairs * (192 + 128)}


# ---------------------------------------------------------------------------- inputs
def _table(g, pages_of, num_pages, width):
    """A block table whose rows take pages of a random permutation of the pool, -1 behind."""
    order = torch.randperm(num_pages, generator=g, device=DEV).int()
    count = torch.tensor(pages_of, device=DEV)
    col = torch.arange(width, device=DEV)
    used = col[None, :] < count[:, None]
    rank = (torch.cumsum(used.flatten(), 0) - 1).clamp(min=0).view(used.shape)
    return torch.where(used, order[rank], -1).int().contiguous()


def _starts(n):
    return torch.tensor([0] + n, device=DEV).cumsum(0).int()


def _angles(positions, rot, base=10000.0):
    """cos | sin of every position's angles, float32 [positions][rot]."""
    freq = base ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    angle = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), 1).float()


def _projected(g, n, width, dtype):
    """Rows of a projection's output, a few channels much larger than the rest."""
    x = torch.randn((n, width), generator=g, device=DEV)
    x *= 1 + 5 * (torch.rand((width,), generator=g, device=DEV) < 0.03)
    return x.to(dtype)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n, t = _counts(c)
    rows = sum(n)
    s = dict(c=c, n_rows=rows, max_n=max(n), max_t=max(t), row_start=_starts(n))
    if c["op"] == "expanded":
        s["key_start"] = _starts(t)
        s["q"] = torch.randn((rows, c["Hq"], 192), generator=g, device=DEV, dtype=torch.bfloat16)
        # the expansion's output: K (without the rotated part) and V of every head side by side
        kv = torch.randn((sum(t), c["Hq"], 256), generator=g, device=DEV, dtype=torch.bfloat16)
        s["k"], s["v"] = kv[..., :128], kv[..., 128:]
        s["r"] = torch.randn((sum(t), DR), generator=g, device=DEV, dtype=torch.bfloat16)
        if own:
            from top_hs2_fa_gb300 import hs2

            s["ws"] = torch.empty(hs2.hs2_latent_prefill_workspace(rows, c["Hq"], c["batch"], s["max_n"], s["max_t"]),
                                  device=DEV, dtype=torch.uint8)
        return s
    pages_of = [-(-v // PAGE) for v in t]
    num_pages = sum(pages_of) + 3
    s.update(table=_table(g, pages_of, num_pages, max(pages_of)),
             seq_len=torch.tensor(t, device=DEV, dtype=torch.int32))
    if c["op"] == "rotate":
        dtype = torch.bfloat16 if c["rows"] == "bf16" else torch.float32
        kd, qd = c["Hkv"] * c["d"], c["Hq"] * c["d"]
        x = _projected(g, rows, qd + 2 * kd, dtype)  # a fused projection's output
        s["q"] = x[:, :qd].unflatten(1, (c["Hq"], c["d"]))
        s["k_rows"] = x[:, qd:qd + kd].unflatten(1, (c["Hkv"], c["d"]))
        s["v_rows"] = x[:, qd + kd:].unflatten(1, (c["Hkv"], c["d"]))
        s["rot"] = _angles(s["max_t"], c["rot"])
        shape = (num_pages, c["Hkv"], PAGE, c["d"])
        for side in ("k", "v"):
            s[side] = torch.zeros(shape, device=DEV, dtype=torch.bfloat16 if c["dtype"] == "bf16" else torch.uint8)
            if c["dtype"] == "fp8":
                # slab scales as a calibration gives them: near one value, no powers of two
                s[side + "_scale"] = (0.9 + 0.2 * torch.rand(shape[:2], generator=g, device=DEV)) / 16
    else:
        d = c["dc"] + DR
        if c["op"] == "append":
            s["k"] = torch.zeros((num_pages, 1, PAGE, d), device=DEV, dtype=torch.bfloat16)
            x = _projected(g, rows, d, torch.bfloat16)  # the down projection's output: latent and key part
            s["c_rows"], s["r_rows"] = x[:, :c["dc"]], x[:, c["dc"]:]
            s["q_raw"] = torch.randn((rows, c["Hq"], 192), generator=g, device=DEV, dtype=torch.bfloat16)[..., 128:]
            # the queries in the latent space: the latent part is there, the rotated part goes behind it
            s["q"] = torch.zeros((rows, c["Hq"], d), device=DEV, dtype=torch.bfloat16)
            s["rot"] = _angles(s["max_t"], DR)
        else:
            s["k"] = torch.randn((num_pages, 1, PAGE, d), generator=g, device=DEV, dtype=torch.bfloat16)
            s["q"] = torch.randn((rows, c["Hq"], d), generator=g, device=DEV, dtype=torch.bfloat16)
    if own:
        from top_hs2_fa_gb300 import hs2

        s["kv"] = hs2.KV(k=s["k"], v=s.get("v"), block_table=s["table"], seq_len=s["seq_len"], k_scale=s.get("k_scale"),
                         v_scale=s.get("v_scale"))
        if c["op"] == "absorbed":
            s["ws"] = torch.empty(hs2.hs2_latent_chunk_workspace(rows, c["Hq"], s["kv"], s["max_n"], s["max_t"]),
                                  device=DEV, dtype=torch.uint8)
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    op = s["c"]["op"]
    if op == "rotate":
        return _rotate_own(s) if own else _rotate_plain(s)
    if op == "append":
        return _append_own(s) if own else _append_plain(s)
    if op == "absorbed":
        return _absorbed_own(s) if own else _absorbed_plain(s)
    return _expanded_own(s) if own else _expanded_plain(s)


def _rotate_own(s):
    from top_hs2_fa_gb300 import hs2

    q = hs2.hs2_kv_write_rot(s["kv"], s["k_rows"], s["v_rows"], s["row_start"], s["rot"], style=s["c"]["style"], q=s["q"])
    k, v = hs2.hs2_kv_read(s["kv"], s["row_start"], s["n_rows"], dtype=torch.bfloat16)
    return {"q": q, "k": k, "v": v}


def _append_own(s):
    from top_hs2_fa_gb300 import hs2

    hs2.hs2_latent_write(s["kv"], s["c_rows"], s["r_rows"], s["row_start"], s["rot"], style=s["c"]["style"],
                         q=s["q_raw"], q_out=s["q"][..., s["c"]["dc"]:])
    c, r = hs2.hs2_latent_read(s["kv"], s["row_start"], s["n_rows"])
    return {"q": s["q"], "c": c, "r": r}


def _absorbed_own(s):
    from top_hs2_fa_gb300 import hs2

    o, lse = hs2.hs2_latent_chunk(s["q"], s["row_start"], s["kv"], _SCALE, s["max_n"], max_t=s["max_t"],
                                  o_dtype=torch.bfloat16, workspace=s["ws"])
    return {"o": o, "lse": lse}


def _expanded_own(s):
    from top_hs2_fa_gb300 import hs2

    o, lse = hs2.hs2_latent_prefill(s["q"], s["k"], s["r"], s["v"], s["row_start"], s["key_start"], _SCALE,
                                    s["max_n"], s["max_t"], o_dtype=torch.bfloat16, workspace=s["ws"])
    return {"o": o, "lse": lse}


def _positions(s):
    """(sequence, position) of every row."""
    start = s["row_start"].long()
    row = torch.arange(s["n_rows"], device=start.device)
    b = torch.bucketize(row, start[1:], right=True)
    return b, s["seq_len"].long()[b] - (start[1:] - start[:-1])[b] + row - start[b]


def _turn(x, at, rot, style):
    """float32 rows x [n][heads][d], the first channels of each head rotated by the positions."""
    half = rot.shape[1] // 2
    cos, sin = rot[at, None, :half], rot[at, None, half:]
    a, b = (x[..., :half], x[..., half:2 * half]) if style == "halves" else (x[..., 0:2 * half:2], x[..., 1:2 * half:2])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat((a, b), -1) if style == "halves" else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _nearest(a, borders):
    """How many of `borders` lie below `a`; on a border the even count of the two."""
    below, upto = torch.bucketize(a, borders, out_int32=True), torch.bucketize(a, borders, right=True, out_int32=True)
    return torch.where(below % 2 == 0, below, upto)


def _e4m3_values():
    """The 127 finite non-negative E4M3 values, ascending by code, in 64 bits."""
    c = torch.arange(127, device=DEV)
    e, m = (c >> 3).double(), (c & 7).double()
    return torch.where(c < 8, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e - 7))


def _rotate_plain(s):
    c = s["c"]
    b, at = _positions(s)
    page, line = s["table"][b, at // PAGE].long(), at % PAGE
    out = {"q": _turn(s["q"].float(), at, s["rot"], c["style"]).to(torch.bfloat16)}
    for side in ("k", "v"):
        x = s[side + "_rows"].float()
        x = _turn(x, at, s["rot"], c["style"]) if side == "k" else x
        if c["dtype"] == "bf16":
            s[side][page, :, line] = x.to(torch.bfloat16)
            out[side] = s[side][page, :, line]
            continue
        scale, e4m3 = s[side + "_scale"][page][..., None], _e4m3_values()
        code = _nearest((x.double() / scale.double()).abs(), (e4m3[1:] + e4m3[:-1]) / 2)  # ties have to be seen exactly
        s[side][page, :, line] = torch.where(x.signbit(), code + 128, code).to(torch.uint8)
        out[side] = (s[side][page, :, line].view(torch.float8_e4m3fn).float() * scale).to(torch.bfloat16)
    return out


def _append_plain(s):
    c = s["c"]
    b, at = _positions(s)
    page, line = s["table"][b, at // PAGE].long(), at % PAGE
    r = _turn(s["r_rows"].float()[:, None], at, s["rot"], c["style"])[:, 0]
    s["k"][page, 0, line] = torch.cat((s["c_rows"], r.to(torch.bfloat16)), 1)
    s["q"][..., c["dc"]:] = _turn(s["q_raw"].float(), at, s["rot"], c["style"]).to(torch.bfloat16)
    stored = s["k"][page, 0, line]
    return {"q": s["q"], "c": stored[:, :c["dc"]], "r": stored[:, c["dc"]:]}


def _padded(s, length):
    """(sequence, token) of every row, rows by (sequence, token) clamped, position of each (sequence, token)."""
    start = s["row_start"].long()
    n = start[1:] - start[:-1]
    row = torch.arange(s["n_rows"], device=start.device)
    b = torch.bucketize(row, start[1:], right=True)
    tok = torch.arange(s["max_n"], device=start.device)
    slot = (start[:-1, None] + tok).clamp(max=s["n_rows"] - 1)
    return b, row - start[b], slot, (length - n)[:, None] + tok


def _softmax(x, at):
    """Weights of the causal softmax of logits x [B][heads][token][T] in place, and its log-sum [B][heads][token]."""
    key = torch.arange(x.shape[-1], device=x.device)
    x.masked_fill_((key > at[..., None])[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    return x.div_(total), (m + torch.log(total)).squeeze(-1)


def _absorbed_plain(s):
    c = s["c"]
    b, i, slot, at = _padded(s, s["seq_len"].long())
    # entries behind a table's end are page 0's: their weight is 0, and so is what they add
    k = s["k"][s["table"].clamp(min=0).long(), 0].flatten(1, 2).float()  # [B, T, dc + 64]
    q = s["q"][slot].float().transpose(1, 2)  # [B, Hq, top, dc + 64]
    x = (q.flatten(1, 2) @ k.transpose(1, 2)).mul_(_SCALE).unflatten(1, q.shape[1:3])
    p, lse = _softmax(x, at)
    o = (p.flatten(1, 2) @ k[..., :c["dc"]]).unflatten(1, q.shape[1:3])
    return {"o": o.transpose(1, 2)[b, i].to(torch.bfloat16), "lse": lse.transpose(1, 2)[b, i]}


def _expanded_plain(s):
    start = s["key_start"].long()
    length = start[1:] - start[:-1]
    b, i, slot, at = _padded(s, length)
    key = (start[:-1, None] + torch.arange(s["max_t"], device=start.device)).clamp(max=s["r"].shape[0] - 1)
    q = s["q"][slot].float().transpose(1, 2)  # [B, Hq, top, 192]
    x = q[..., :128] @ s["k"][key].float().permute(0, 2, 3, 1)
    x += q[..., 128:] @ s["r"][key].float().transpose(1, 2)[:, None]
    p, lse = _softmax(x.mul_(_SCALE), at)
    o = p @ s["v"][key].float().transpose(1, 2)
    return {"o": o.transpose(1, 2)[b, i].to(torch.bfloat16), "lse": lse.transpose(1, 2)[b, i]}


# ---------------------------------------------------------------------------- 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rotate":
        return _rotate_exact(s)
    if c["op"] == "append":
        return _append_exact(s)
    return _attend_exact(s)


def _turn64(x, s):
    """Rows x [n][heads][d] rotated one sequence after another, every pair as a complex number."""
    x, start, rot = x.double().clone(), s["row_start"].tolist(), s["rot"].double()
    half, lengths = rot.shape[1] // 2, s["seq_len"].tolist()
    for b, t in enumerate(lengths):
        lo, hi = start[b], start[b + 1]
        z = torch.complex(rot[t - (hi - lo):t, :half], rot[t - (hi - lo):t, half:])[:, None]
        part = x[lo:hi, :, :2 * half]
        if s["c"]["style"] == "halves":
            w = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * z
            x[lo:hi, :, :2 * half] = torch.cat((w.real, w.imag), -1)
        else:
            w = torch.view_as_complex(part.unflatten(-1, (half, 2)).contiguous()) * z
            x[lo:hi, :, :2 * half] = torch.view_as_real(w).flatten(-2)
    return x


def _rotate_exact(s):
    c, out = s["c"], {"q": _turn64(s["q"], s)}
    start, lengths = s["row_start"].tolist(), s["seq_len"].tolist()
    page = torch.cat([s["table"][b, torch.arange(t - (start[b + 1] - start[b]), t, device=DEV) // PAGE]
                      for b, t in enumerate(lengths)]).long()
    for side in ("k", "v"):
        x = _turn64(s["k_rows"], s) if side == "k" else s["v_rows"].double()
        if c["dtype"] == "fp8":
            slab = s[side + "_scale"][page].double()[..., None]
            a = (x / slab).abs()
            # spacing of the E4M3 values about a: 3 mantissa bits, exponents from -6 on
            step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
            x = x.sign() * (torch.round(a / step) * step).clamp(max=448) * slab
        out[side] = x
    return out


def _append_exact(s):
    c = s["c"]
    q = s["q"].double()
    q[..., c["dc"]:] = _turn64(s["q_raw"], s)
    return {"q": q, "c": s["c_rows"].double(), "r": _turn64(s["r_rows"][:, None], s)[:, 0]}


def _attend_exact(s):
    c = s["c"]
    start = s["row_start"].tolist()
    dv = c["dc"] if c["op"] == "absorbed" else 128
    o = torch.empty((*s["q"].shape[:2], dv), device=DEV, dtype=torch.float64)
    lse = torch.empty(s["q"].shape[:2], device=DEV, dtype=torch.float64)
    begin = s["key_start"].tolist() if c["op"] == "expanded" else None
    for b in range(c["batch"]):
        lo, hi = start[b], start[b + 1]
        if begin is None:
            t = int(s["seq_len"][b])
            shared = s["k"][s["table"][b, :-(-t // PAGE)].long()].flatten(0, 2)[:t].double()
        else:
            t = begin[b + 1] - begin[b]
            shared = s["r"][begin[b]:begin[b + 1]].double()
        pos = torch.arange(t - (hi - lo), t, device=DEV)[:, None]
        seen = torch.arange(t, device=DEV)[None, :] <= pos
        for h in range(c["Hq"]):
            if begin is None:
                k, v = shared, shared[:, :dv]
            else:
                k = torch.cat((s["k"][begin[b]:begin[b + 1], h].double(), shared), 1)
                v = s["v"][begin[b]:begin[b + 1], h].double()
            x = torch.where(seen, s["q"][lo:hi, h].double() @ k.T / math.sqrt(192), -math.inf)
            z = torch.logsumexp(x, 1)
            o[lo:hi, h] = torch.exp(x - z[:, None]) @ v
            lse[lo:hi, h] = z
    return {"o": o, "lse": lse}
