"""Workloads of the 8-bit resident KV cache: writing tokens into it, reading
them back, and attention over it.

The cache holds FP8 E4M3FN or INT8 codes of K and V in pages of T tokens, with
one FP32 scale for each (page, KV head) of K and one of V:
    k_codes [pages, H, T, D], v_codes [pages, H, D, T] (V token-minor),
    k_scales, v_scales [pages, H].
A batch names its sequences by a block table [seqs, columns] of page ids, by
cu_rows [seqs + 1] (rows cu_rows[b] .. cu_rows[b+1] - 1 of the row tensors are
sequence b's) and by lengths [seqs]: with n rows, sequence b's rows are its
positions lengths[b] - n .. lengths[b] - 1.

write   quantises the rows of k and v into their pages.  A page whose first
        token is written takes the scale of the new tokens' largest |x|; a
        page that is appended to keeps its scale unless a new token needs a
        larger one, and then its earlier codes are quantised anew.
read    gives the rows back: code * scale, rounded to the rows' type.
attend  softmax(scale * q k^T) v over the positions a row may see (causal:
        those up to its own; window w: the last w of them), with the log of
        each softmax's sum.  H query heads in groups share a KV head.

With `own` false the plain forms run (elementary torch operations in 32
bits); with `own` true, the library's calls.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


def listed():
    # H = 8, D = 128, T = 16 is the repository's Llama-3-8B and Qwen3-8B cache
    # shape (32 query heads: 4 to a KV head); H = 1 is its 8-way
    # tensor-parallel shard; D = 64 and 256 come from its head-size sweep.
    base = dict(kv_heads=8, group=4, dim=128, page=16, causal=True, window=0)
    return [
        # one user's next token, appended to a half-filled page
        dict(base, name="write_token", op="write", codec="fp8", type="bf16", seqs=1, rows=1, rows_to=1, past=700,
             past_to=700),
        # a serving step's tokens, one for each of 256 users
        dict(base, name="write_step", op="write", codec="int8", type="bf16", seqs=256, rows=1, rows_to=1, past=1,
             past_to=4000),
        # prompts of many lengths, some of them continued, on a small model's cache
        dict(base, name="write_prompts", op="write", codec="fp8", type="fp16", seqs=24, rows=100, rows_to=6000, past=0,
             past_to=45, kv_heads=4, dim=64, page=32),
        # the benchmark's 64K tokens brought into the cache in one call
        dict(base, name="write_bulk", op="write", codec="int8", type="bf16", seqs=8, rows=8192, rows_to=8192, past=0,
             past_to=0),
        # the last tokens of a few sequences, for a check or a draft model
        dict(base, name="read_tail", op="read", codec="fp8", type="fp16", seqs=5, rows=37, rows_to=311, past=90,
             past_to=2000, kv_heads=4, dim=256, page=64),
        # 64K tokens back into 16 bits, before they are encoded for the host tier
        dict(base, name="read_bulk", op="read", codec="fp8", type="bf16", seqs=8, rows=8000, rows_to=8400, past=0,
             past_to=0),
        # one user's next token: nothing but latency
        dict(base, name="attend_one", op="attend", codec="fp8", type="bf16", seqs=1, rows=1, rows_to=1, past=999,
             past_to=999),
        # a serving step: 64 users, one token each, ragged lengths
        dict(base, name="attend_step", op="attend", codec="fp8", type="bf16", seqs=64, rows=1, rows_to=1, past=500,
             past_to=8000),
        # few users with very long contexts on one shard's KV head
        dict(base, name="attend_long", op="attend", codec="int8", type="bf16", seqs=3, rows=1, rows_to=1, past=100000,
             past_to=131071, kv_heads=1),
        # five drafted tokens a user are checked, with a sliding window
        dict(base, name="attend_draft", op="attend", codec="int8", type="fp16", seqs=16, rows=5, rows_to=5, past=300,
             past_to=5000, kv_heads=4, group=7, dim=64, page=64, window=1024),
        # chunks of prompts behind what is cached already
        dict(base, name="attend_chunk", op="attend", codec="int8", type="fp16", seqs=6, rows=300, rows_to=2100, past=0,
             past_to=6000),
        # one long prompt, the heaviest call
        dict(base, name="attend_prompt", op="attend", codec="fp8", type="bf16", seqs=1, rows=8192, rows_to=8192, past=0,
             past_to=0),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        c = dict(op=rng.choice(("write", "read", "attend", "attend")), codec=rng.choice(("fp8", "int8")),
                 type=rng.choice(("bf16", "fp16")), kv_heads=rng.choice((1, 2, 3, 4, 8)), group=rng.choice((1, 2, 4, 5, 7, 8)),
                 dim=rng.choice((32, 64, 128, 256)), page=rng.choice((16, 32, 64, 128)), causal=True, window=0)
        if c["op"] != "attend":
            c["seqs"] = spread(1, 256)
            c["rows"] = 1 if rng.random() < 0.3 else spread(1, 8192)
            c["rows_to"] = c["rows"] if rng.random() < 0.3 else spread(c["rows"], 4 * c["rows"])
            c["past"] = spread(1, 4000) - 1
            c["past_to"] = spread(c["past"] + 1, 4000) - 1
        elif rng.random() < 0.5:       # single tokens and drafts
            c["seqs"] = spread(1, 128)
            c["rows"] = c["rows_to"] = rng.choice((1, 1, 1, 2, 3, 5, 8))
            c["past"] = spread(1, 131072) - 1
            c["past_to"] = spread(c["past"] + 1, 131072) - 1
        else:                          # prompts and chunks
            c["seqs"] = spread(1, 16)
            c["rows"] = spread(16, 8192)
            c["rows_to"] = spread(c["rows"], 8192)
            c["past"] = 0 if rng.random() < 0.5 else spread(1, 8192)
            c["past_to"] = spread(c["past"] + 1, 8192)
        if c["op"] == "attend":
            c["causal"] = rng.random() < 0.9
            c["window"] = spread(64, 4096) if rng.random() < 0.25 else 0
        rows, past = sizes(c)
        total, longest = int(rows.sum()), int((rows + past).max())
        most = 8192 * 8 * 128 * 8                           # elements of 64K tokens of K at H = 8, D = 128
        if c["op"] != "attend" and (total * c["kv_heads"] * c["dim"] > most
                                    or int((rows + past).sum()) * c["kv_heads"] * c["dim"] > 2 * most):
            continue
        heads = c["kv_heads"] * c["group"]
        scores = c["seqs"] * int(rows.max()) * longest * heads
        if c["op"] == "attend" and (scores > 8192 * 8192 * 32 or scores * c["dim"] > 8192 * 8192 * 32 * 128 // 2
                                    or c["seqs"] * longest * c["kv_heads"] * c["dim"] > most * 8):
            continue
        return c


# ------------------------------------------------------------------ inputs
def sizes(c):
    """Rows and earlier tokens of each sequence: spread from `rows` to `rows_to` and from `past` to `past_to` in a
    fixed order that looks random."""
    b = np.arange(c["seqs"])
    u, w = (b * 0.6180339887 + 0.37) % 1.0, (b * 0.7548776662 + 0.11) % 1.0
    rows = np.rint(c["rows"] + (c["rows_to"] - c["rows"]) * u).astype(np.int64)
    past = np.rint(c["past"] + (c["past_to"] - c["past"]) * w).astype(np.int64)
    return rows, past


def quantise(x, scale, codec):
    """Codes of x against scale: E4M3FN or INT8, to nearest, ties to even, values clipped to the type's range."""
    t = x / scale
    if codec == "fp8":
        return t.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return torch.round(t).clamp(-127.0, 127.0).to(torch.int8)


def scale_of(amax, codec):
    a = amax.clamp_min(float(np.float32(1e-12)))
    if codec == "fp8":
        return a * torch.full_like(a, 1.0 / 448.0)
    return a / torch.full_like(a, 127.0)           # a tensor: a number would be multiplied by its reciprocal


def _floats(gen, shape, channel):
    """N(0, 1) values, with a lognormal size for each channel of K."""
    x = torch.randn(shape, generator=gen, device=DEV)
    return x * torch.exp(torch.randn((shape[1], 1, shape[3]), generator=gen, device=DEV)) if channel else x


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7919 + 11)
    rows, past = sizes(c)
    B, H, D, T, dt = c["seqs"], c["kv_heads"], c["dim"], c["page"], TYPES[c["type"]]
    lengths = rows + past
    n, pages = int(rows.sum()), -(-lengths // T)
    P = int(pages.sum()) + 3
    perm = torch.randperm(P, generator=gen, device=DEV).to(torch.int32)
    cols = int(pages.max())
    first = torch.as_tensor(np.cumsum(pages) - pages, device=DEV)
    col = torch.arange(cols, device=DEV)[None, :]
    inside = col < torch.as_tensor(pages, device=DEV)[:, None]
    table = torch.where(inside, perm[(first[:, None] + col).clamp_max(P - 1)], -1).to(torch.int32).contiguous()
    s = dict(case=c, n=n, most_rows=int(rows.max()), longest=int(lengths.max()), table=table,
             cu=torch.as_tensor(np.concatenate([[0], np.cumsum(rows)]), device=DEV).to(torch.int32),
             lengths=torch.as_tensor(lengths, device=DEV).to(torch.int32))
    for name, channel in (("k", True), ("v", False)):
        x = _floats(gen, (P, H, T, D), channel)
        sc = scale_of(x.abs().amax((2, 3)), c["codec"])
        codes = quantise(x, sc[:, :, None, None], c["codec"])
        s[name + "_codes"] = (codes if name == "k" else codes.transpose(2, 3)).contiguous()
        s[name + "_scales"] = sc
        del x, codes
    if c["op"] == "write":
        # k and v are slices of one projection's output, as an engine has them
        qkv = torch.randn((n, (c["group"] + 2) * H, D), generator=gen, device=DEV)
        qkv[:, c["group"] * H:(c["group"] + 1) * H] *= torch.exp(torch.randn((H, D), generator=gen, device=DEV))
        qkv = qkv.to(dt)
        s["k"], s["v"] = qkv[:, c["group"] * H:(c["group"] + 1) * H], qkv[:, (c["group"] + 1) * H:]
    elif c["op"] == "attend":
        s["q"] = torch.randn((n, H * c["group"], D), generator=gen, device=DEV).to(dt)
    if own:                                        # what a user's program keeps: the handles and its buffers
        import kv_cache_page_kvc_amd as kvc
        s["cache"] = kvc.Cache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
        s["batch"] = kvc.Batch(s["table"], s["cu"], s["lengths"], n, s["most_rows"], s["longest"])
        if c["op"] == "write":
            s["args"] = kvc.Rows(s["k"]), kvc.Rows(s["v"])
        elif c["op"] == "read":
            s["out"] = tuple(torch.empty((n, H, D), dtype=dt, device=DEV) for _ in range(2))
            s["args"] = kvc.Rows(s["out"][0]), kvc.Rows(s["out"][1])
        else:
            s["out"] = torch.empty_like(s["q"]), torch.empty((n, H * c["group"]), device=DEV)
            s["options"] = kvc.Attend(H * c["group"], causal=c["causal"], window=c["window"])
            need = kvc.kvc_plan_attend(s["cache"], s["batch"], s["options"])
            s["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
            s["args"] = kvc.Rows(s["q"]), kvc.Rows(s["out"][0]), s["out"][1]
        s["stream"] = torch.cuda.current_stream().cuda_stream
        s["ctx"] = context()
    return s


_context = None


def context():
    global _context
    if _context is None:
        import kv_cache_page_kvc_amd as kvc
        _context = kvc.kvc_create(torch.cuda.current_device(), 0)
    return _context


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        import kv_cache_page_kvc_amd as kvc
        if op == "write":
            kvc.kvc_cache_write(s["ctx"], s["cache"], s["batch"], *s["args"], s["stream"])
        elif op == "read":
            kvc.kvc_cache_read(s["ctx"], s["cache"], s["batch"], *s["args"], s["stream"])
        else:
            kvc.kvc_cache_attend(s["ctx"], s["cache"], s["batch"], s["options"], *s["args"], s["workspace"], s["stream"])
    else:
        s["out"] = plain_write(s) if op == "write" else plain_read(s) if op == "read" else plain_attend(s)
    if op == "write":
        return {x: s[x] for x in ("k_codes", "v_codes", "k_scales", "v_scales")}
    return dict(zip(("k", "v") if op == "read" else ("out", "lse"), s["out"]))


def places(s):
    """Page and place in the page of every row."""
    T, cu = s["case"]["page"], s["cu"].long()
    row = torch.arange(s["n"], device=DEV)
    b = torch.searchsorted(cu, row, right=True) - 1
    pos = s["lengths"].long()[b] - cu[b + 1] + row
    return s["table"][b, pos // T].long(), pos % T


def plain_write(s):
    c = s["case"]
    page, at = places(s)
    touched, where = torch.unique(page, return_inverse=True)
    T = c["page"]
    low = torch.full((touched.numel(),), T, dtype=torch.int64, device=DEV).scatter_reduce_(0, where, at, "amin")
    fresh = (low == 0)[:, None]
    kept = (torch.arange(T, device=DEV)[None, :] < low[:, None]) & ~fresh
    plain_write_one(s, "k", page, at, touched, where, fresh, kept)
    plain_write_one(s, "v", page, at, touched, where, fresh, kept)


def plain_write_one(s, name, page, at, touched, where, fresh, kept):
    codec, x = s["case"]["codec"], s[name].float()
    codes, scales = s[name + "_codes"], s[name + "_scales"]
    codes = codes if name == "k" else codes.transpose(2, 3)                                   # [P, H, T, D]
    amax = torch.zeros((touched.numel(), x.shape[1]), device=DEV)
    amax = amax.scatter_reduce_(0, where[:, None].expand(-1, x.shape[1]), x.abs().amax(2), "amax")
    need, old = scale_of(amax, codec), scales[touched]
    new = torch.where(fresh, need, torch.maximum(old, need))
    grown = kept[:, None, :] & (new > old)[:, :, None]                                       # [touched, H, T]
    at_p, at_h, at_t = torch.nonzero(grown, as_tuple=True)
    earlier = codes[touched[at_p], at_h, at_t].float() * old[at_p, at_h, None]
    codes[touched[at_p], at_h, at_t] = quantise(earlier, new[at_p, at_h, None], codec)
    scales[touched] = new
    codes[page, :, at] = quantise(x, new[where][:, :, None], codec)


def plain_read(s):
    page, at = places(s)
    dt = TYPES[s["case"]["type"]]
    k = s["k_codes"][page, :, at].float() * s["k_scales"][page][:, :, None]
    v = s["v_codes"][page, :, :, at].float() * s["v_scales"][page][:, :, None]
    return k.to(dt), v.to(dt)


def plain_attend(s):
    c = s["case"]
    B, H, G, D, T = c["seqs"], c["kv_heads"], c["group"], c["dim"], c["page"]
    R, cu, length = s["most_rows"], s["cu"].long(), s["lengths"].long()
    pages = s["table"].long().clamp_min(0)                                                    # [B, columns]
    L = pages.shape[1] * T
    k = (s["k_codes"][pages].float() * s["k_scales"][pages][..., None, None])                 # [B, columns, H, T, D]
    k = k.permute(0, 2, 4, 1, 3).reshape(B * H, D, L)
    v = (s["v_codes"][pages].float() * s["v_scales"][pages][..., None, None])                 # [B, columns, H, D, T]
    v = v.permute(0, 2, 1, 4, 3).reshape(B * H, L, D)
    rows = torch.arange(R, device=DEV)
    real = rows[None, :] < (cu[1:] - cu[:-1])[:, None]                                        # [B, R]
    at = (cu[:-1, None] + rows[None, :]).clamp_max(s["n"] - 1)
    q = s["q"].float()[at].reshape(B, R, H, G, D).permute(0, 2, 3, 1, 4).reshape(B * H, G * R, D)
    pos = (length - cu[1:] + cu[:-1])[:, None] + rows[None, :]                                # [B, R]
    j = torch.arange(L, device=DEV)
    seen = (j < length[:, None, None]) & real[:, :, None]                                     # [B, R, L]
    if c["causal"]:
        seen &= j <= pos[:, :, None]
    if c["window"]:
        seen &= j > pos[:, :, None] - c["window"]
    p = torch.bmm(q, k).mul_(1.0 / math.sqrt(D)).reshape(B, H * G, R, L)
    p.masked_fill_(~seen[:, None], -math.inf)
    most = p.amax(3, keepdim=True)
    most = torch.where(most == -math.inf, torch.zeros_like(most), most)
    p = p.sub_(most).exp_()
    total = p.sum(3, keepdim=True)
    out = torch.bmm(p.reshape(B * H, G * R, L), v).reshape(B, H * G, R, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (most + torch.log(total))[..., 0]
    return out.transpose(1, 2)[real].to(TYPES[c["type"]]), lse.transpose(1, 2)[real]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    rows, past = sizes(c)
    vec = c["kv_heads"] * c["dim"]
    n, length = int(rows.sum()), rows + past
    touched = int(((length + c["page"] - 1) // c["page"] - past // c["page"]).sum())
    if c["op"] != "attend":                        # rows in 16 bits, their codes, the touched pages' scales
        return {"bytes": 2.0 * n * vec * 3 + 8.0 * touched * c["kv_heads"], "flops": 2.0 * 3 * n * vec}
    i = [past[b] + np.arange(rows[b]) for b in range(c["seqs"])]
    last = [np.minimum(p, l - 1) if c["causal"] else np.full(len(p), l - 1) for p, l in zip(i, length)]
    begin = [np.maximum(0, p - c["window"] + 1) if c["window"] else np.zeros_like(p) for p in i]
    pairs = sum(int((l - f + 1).sum()) for l, f in zip(last, begin))
    read = sum(int(l.max() - f.min() + 1) for l, f in zip(last, begin))
    heads = c["kv_heads"] * c["group"]
    return {"bytes": 2.0 * read * vec + 8.0 * read / c["page"] * c["kv_heads"] + n * heads * (4.0 * c["dim"] + 4),
            "flops": 4.0 * pairs * heads * c["dim"]}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    cu, lengths = s["cu"].tolist(), s["lengths"].tolist()
    values = {}
    for name in ("k", "v"):
        x = s[name + "_codes"].double() * s[name + "_scales"].double()[:, :, None, None]
        values[name] = x if name == "k" else x.transpose(2, 3)                                # [P, H, T, D]
    parts = [_exact_one(s, c, values, b, cu[b], cu[b + 1], lengths[b]) for b in range(c["seqs"])]
    if c["op"] != "write":
        return {x: torch.cat([p[x] for p in parts]) for x in parts[0]}
    whole = {}
    for name in ("k", "v"):
        sc = s[name + "_scales"].double()
        codes = s[name + "_codes"].double()
        codes = codes if name == "k" else codes.transpose(2, 3)
        for p in parts:
            page, new, put = p[name]
            sc[page] = new
            codes[page] = torch.where(torch.isnan(put), codes[page], put)
        whole[name + "_scales"] = sc
        # INT8 codes are whole numbers: their ties go by the 32-bit quotient, which 64 bits do not tell
        whole[name + "_codes"] = None if c["codec"] == "int8" else codes if name == "k" else codes.transpose(2, 3)
    return whole


def _exact_one(s, c, values, b, r0, r1, length):
    T, n = c["page"], r1 - r0
    page = s["table"][b].long()
    page = page[:-(-length // T)]
    start = length - n
    if c["op"] == "write":
        return {x: _exact_write(s, c, x, page, r0, n, start, length) for x in ("k", "v")}
    kv = {x: values[x][page].transpose(1, 2).reshape(-1, c["kv_heads"], c["dim"])[:length] for x in ("k", "v")}
    if c["op"] == "read":
        return {x: kv[x][start:] for x in kv}
    q = s["q"][r0:r1].double().reshape(n, c["kv_heads"], c["group"], c["dim"])
    pos = torch.arange(start, length, device=DEV)[:, None]
    j = torch.arange(length, device=DEV)[None, :]
    hidden = torch.zeros((n, length), dtype=torch.bool, device=DEV)
    if c["causal"]:
        hidden = hidden | (j > pos)
    if c["window"]:
        hidden = hidden | (j <= pos - c["window"])
    out, lse = [], []
    for h in range(c["kv_heads"]):                 # one KV head at a time: the scores fit beside the rest
        sc = torch.matmul(q[:, h].transpose(0, 1), kv["k"][:, h].t().contiguous()) / math.sqrt(c["dim"])   # [G, n, L]
        sc = sc.masked_fill(hidden, -math.inf)
        z = torch.logsumexp(sc, 2)
        p = torch.softmax(sc, 2)
        p = torch.where(torch.isnan(p), torch.zeros_like(p), p)
        out.append(torch.matmul(p, kv["v"][:, h].contiguous()).transpose(0, 1))
        lse.append(z.transpose(0, 1))
    return {"out": torch.stack(out, 1).reshape(n, -1, c["dim"]), "lse": torch.stack(lse, 1).reshape(n, -1)}


def _e4m3(t):
    """The nearest E4M3FN value, ties to even."""
    t = t.clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(t / step) * step


def _exact_write(s, c, name, page, r0, n, start, length):
    """Pages from the one that holds `start` on: their new scales and codes (NaN where a code stays)."""
    T, H, D, top = c["page"], c["kv_heads"], c["dim"], 448.0 if c["codec"] == "fp8" else 127.0
    rnd = _e4m3 if c["codec"] == "fp8" else (lambda t: torch.round(t).clamp(-127, 127))
    page = page[start // T:]
    m, off = page.numel(), start % T
    x = torch.full((m * T, H, D), math.nan, dtype=torch.float64, device=DEV)
    x[off:off + n] = s[name][r0:r0 + n].double()
    x = x.reshape(m, T, H, D).transpose(1, 2)                                                 # [m, H, T, D]
    need = torch.nan_to_num(x).abs().amax((2, 3)).clamp_min(1e-12) / top
    old = s[name + "_scales"][page].double()
    new = need.clone()
    codes = s[name + "_codes"][page].double()
    codes = codes if name == "k" else codes.transpose(2, 3)
    if off:
        # the scales are FP32 values: one that 64 bits find larger by less than a rounding is not larger
        grows = need[0].float() > old[0].float()
        new[0] = torch.where(grows, need[0], old[0])
        x[0, :, :off] = torch.where(grows[:, None, None], codes[0, :, :off] * old[0][:, None, None], math.nan)
    return page, new, rnd(x / new[:, :, None, None])
