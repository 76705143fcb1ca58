"""The operators of a paged key-value cache held in few bits, as they are
measured: rows quantized as they are written into its pages, rows read back,
and the attention of one new token per sequence over it.

`run` computes one pass: with `own` false in plain torch operations (fp32
arithmetic whatever the inputs' type), with `own` true through
learnable_butterfly_rotation_amd.  `exact` gives the same outputs from the
definitions in fp64.

A cache holds pages of `page` tokens of `kv` heads of `d` elements, keys and
values alike, as bf16, int8, e4m3 or int4 (two codes to a byte, element 2i in
the low half); each head's row of a token in 8 or 4 bits has one fp16 scale:
scale = fp16(max |x| / top), code = rnd(x / scale), top = 127, 448 or 7.  The
cases differ in `kind`:

* write: the rows of `tokens` tokens into given slots (page * size + place);
  a slot of -1 is a padded row, which is left out;
* store: the same, and the rows read back from where they were written;
* read: the rows of given slots;
* attend: y = sum_t p_t v_t with p = softmax(scale * k_t . q) over the tokens
  of the row's sequence, heads / kv query heads to a key-value head; a row of
  length 0 (a padded batch) gives 0;
* step: a layer's decode step: the new tokens' rows written, then attend, with
  q, k and v as they lie in the projection's output.
"""
import math

import torch

own = False

_BF16, _F32 = "bf16", "f32"
_TYPES = {_BF16: torch.bfloat16, _F32: torch.float32}
_PAGES = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn,
          "int4": torch.uint8}
_TOP = {"int8": 127.0, "e4m3": 448.0, "int4": 7.0}
_ELEMENT = {"bf16": 2.0, "int8": 1.0, "e4m3": 1.0, "int4": 0.5}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def _attend(rows, heads, kv, d, length, page, fmt, q=_BF16, y=_BF16, pad=0, window=0, lse=False,
            kind="attend"):
    return {"kind": kind, "rows": rows, "heads": heads, "kv": kv, "d": d, "length": length,
            "page": page, "format": fmt, "q": q, "y": y, "pad": pad, "window": window, "lse": lse}


def _rows(kind, tokens, kv, d, page, fmt, x, padded=False):
    return {"kind": kind, "tokens": tokens, "kv": kv, "d": d, "page": page, "format": fmt, "x": x,
            "padded": padded}


def listed():
    return [
        # one sequence, a few hundred tokens: latency is all that counts
        dict(_attend(1, 32, 8, 128, 321, 16, "int8"), name="attend_token_int8"),
        # a few conversations of a model of 32 full heads (4096 wide), 4 bits
        dict(_attend(5, 32, 32, 128, 1023, 16, "int4"), name="attend_chat_int4"),
        # a full serving batch of ragged lengths with three padded rows
        dict(_attend(64, 32, 8, 128, 8192, 64, "int4", pad=3), name="attend_batch_int4"),
        # one very long document
        dict(_attend(1, 32, 8, 128, 131072, 256, "e4m3"), name="attend_long_e4m3"),
        # sliding-window layer, one key-value head of 256 for 16 query heads,
        # the cache unquantized
        dict(_attend(24, 16, 1, 256, 5000, 32, "bf16", window=2047), name="attend_window_bf16"),
        # fp32 rows of short heads, with the log-sum that joins two caches
        dict(_attend(9, 64, 16, 64, 2000, 32, "int8", q=_F32, y=_F32, lse=True),
             name="attend_f32_int8"),
        # a decode step of 32 sequences: the new rows written, then read
        dict(_attend(32, 32, 8, 128, 4096, 64, "int8", kind="step"), name="step_int8"),
        # the new rows of a decode batch, some of it padded
        dict(_rows("write", 16, 32, 128, 16, "e4m3", _BF16, True), name="write_tokens_e4m3"),
        # a prompt of 8192 tokens
        dict(_rows("write", 8192, 8, 128, 64, "int8", _BF16), name="write_prompt_int8"),
        # an fp32 prompt of a model 5120 wide (40 heads), written and read back
        dict(_rows("store", 4099, 40, 128, 32, "int4", _F32), name="store_prompt_int4"),
        # a long shared prefix read back for a prefill over it
        dict(_rows("read", 32768, 8, 128, 64, "int4", _BF16), name="read_prefix_int4"),
        # a few rows of short heads
        dict(_rows("read", 77, 4, 64, 16, "bf16", _F32), name="read_rows_bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "step", "write", "store", "read"])
    fmt = rng.choice(["bf16", "int8", "e4m3", "int4", "int4"])
    d = rng.choice([64, 128, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    kv = rng.choice([1, 2, 4, 8, 8, 16, 32, rng.randrange(1, 41)])
    if kind in ("attend", "step"):
        share = rng.choice([1, 1, 2, 4, 4, 8, 16, 5, 7, 20])
        share = max(1, min(share, 64 // kv))
        rows = _log_int(rng, 1, 128)
        # at most as much cache as the largest listed case reads, padded lengths counted
        most = int((1 << 27) / (rows * kv * d * _ELEMENT[fmt]))
        length = _log_int(rng, 1, max(1, min(65536, most)))
        window = rng.choice([0, 0, 0, _log_int(rng, 1, length)]) if kind == "attend" else 0
        q = _BF16 if kind == "step" else rng.choice([_BF16, _BF16, _F32])
        return _attend(rows, kv * share, kv, d, length, page, fmt, q=q,
                       y=rng.choice([_BF16, _BF16, _F32]), pad=rng.choice([0, 0, rows // 8]),
                       window=window, lse=rng.random() < 0.3, kind=kind)
    if kind == "store":
        fmt = "int4"
    elif kind == "write" and fmt == "int4":
        fmt = "int8"
    tokens = _log_int(rng, 1, min(32768, (1 << 25) // (kv * d)))
    return _rows(kind, tokens, kv, d, page, fmt, rng.choice([_BF16, _F32]), rng.random() < 0.3)


# ---------------------------------------------------------------------------
# what a program has in hand before the call
# ---------------------------------------------------------------------------

def _lengths(case):
    """The tokens of every sequence, the longest first and the padded rows
    last: spread over a factor of sixteen."""
    n, longest = case["rows"], case["length"]
    g = torch.Generator().manual_seed(1000 * n + longest)
    u = torch.rand(n, generator=g, dtype=torch.float64)
    lens = [max(1, int(longest * 16.0 ** (-float(v)))) for v in u]
    lens[0] = longest
    for i in range(case["pad"]):
        lens[n - 1 - i] = 0
    return lens


def _randn(g, shape, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale


def _keys(g, *shape):
    """Rows of unit variance with 2 % of the channels four times as large."""
    x = _randn(g, shape)
    d = shape[-1]
    x[..., torch.randperm(d, generator=g, device="cuda")[: max(1, d // 50)]] *= 4.0
    return x


def _values(g, *shape):
    """Rows whose sizes differ from token to token."""
    return _randn(g, shape) * torch.exp(_randn(g, shape[:-1], 0.5))[..., None]


def _quantized(x, fmt):
    """The codes of rows (the last axis) as numbers, and their fp16 scales;
    the quotients in fp64, since roundings turn on their last bit."""
    scale = (x.abs().amax(-1).double() / _TOP[fmt]).clamp(max=65504.0).to(torch.float16)
    d = scale.double()[..., None]
    q = torch.where(d > 0, x / d, 0.0).clamp(-_TOP[fmt], _TOP[fmt])
    return (q.to(torch.float8_e4m3fn) if fmt == "e4m3" else torch.round(q).to(torch.int8)), scale


def _packed(codes, fmt):
    if fmt != "int4":
        return codes
    u = codes.view(torch.uint8) & 15
    return u[..., 0::2] | (u[..., 1::2] << 4)


def _unpacked(codes, fmt):
    """What the bytes of rows stand for, in fp32."""
    if fmt != "int4":
        return codes.float()
    both = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(*codes.shape[:-1], -1)
    return (both.to(torch.int8) ^ 8).float() - 8.0


def _cache(x, fmt):
    """Pages and scales of rows."""
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    codes, scale = _quantized(x, fmt)
    return _packed(codes, fmt), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    kv, d, page, fmt = case["kv"], case["d"], case["page"], case["format"]
    s = {"case": case}
    empty = lambda dt, *shape: torch.empty(shape, dtype=dt, device="cuda")
    if case["kind"] in ("attend", "step"):
        rows, heads = case["rows"], case["heads"]
        lens = torch.tensor(_lengths(case), device="cuda")
        lens = lens[torch.randperm(rows, generator=g, device="cuda")]
        used = (lens + page - 1) // page
        pages, width = int(used.sum()) + 3, -(-case["length"] // page)
        # every sequence's pages lie anywhere in the pool; the table's rest is -1
        order = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(width, device="cuda")
        ids = order[((used.cumsum(0) - used)[:, None] + at).clamp(max=pages - 1)]
        s["tables"] = torch.where(at < used[:, None], ids, -1).to(torch.int32)
        s["lens"] = lens.to(torch.int32)
        s["y"] = empty(_TYPES[case["y"]], rows, heads, d)
        s["lse"] = empty(torch.float32, rows, heads) if case["lse"] else None
        if case["kind"] == "attend":
            s["q"] = _randn(g, (rows, heads, d), 1.5).to(_TYPES[case["q"]])
        else:
            qkv = _keys(g, rows, heads + 2 * kv, d).to(torch.bfloat16).reshape(rows, -1)
            q, k, v = qkv.split([heads * d, kv * d, kv * d], dim=1)
            s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, d)) for t in (q, k, v))
            last = (lens - 1).clamp(min=0)
            slot = ids.gather(1, (last // page)[:, None])[:, 0] * page + last % page
            s["slots"] = torch.where(lens > 0, slot, -1).to(torch.int32)
    else:
        tokens = case["tokens"]
        width = -(-tokens // page)
        pages = width + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(tokens, device="cuda")
        slots = order[at // page] * page + at % page
        if case["padded"]:
            slots[torch.rand(tokens, generator=g, device="cuda") < 0.125] = -1
        s["slots"] = slots.to(torch.int32)
        t = _TYPES[case["x"]]
        if case["kind"] == "read":
            s["k"], s["v"] = empty(t, tokens, kv, d), empty(t, tokens, kv, d)
        else:
            s["k"] = _keys(g, tokens, kv, d).to(t)
            s["v"] = _values(g, tokens, kv, d).to(t)
        if case["kind"] == "store":
            s["k_out"], s["v_out"] = empty(t, tokens, kv, d), empty(t, tokens, kv, d)
    s["k_cache"], s["k_scales"] = _cache(_keys(g, pages, kv, page, d), fmt)
    s["v_cache"], s["v_scales"] = _cache(_values(g, pages, kv, page, d), fmt)
    if own and case["kind"] in ("attend", "step"):  # scratch that only the framework's call takes
        import learnable_butterfly_rotation_amd as B
        s["workspace"] = torch.empty(
            max(1, B.bfly_cache_attention_workspace_bytes(rows, heads, kv, d, case["length"])),
            dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _write_plain(s):
    c = s["case"]
    at = torch.nonzero(s["slots"] >= 0)[:, 0]
    slots = s["slots"][at].long()
    page, place = slots // c["page"], slots % c["page"]
    for x, cache, scales in ((s["k"], s["k_cache"], s["k_scales"]),
                             (s["v"], s["v_cache"], s["v_scales"])):
        codes, scale = _cache(x[at].float(), c["format"])
        # one byte of e4m3 is moved as a byte
        cache.view(torch.uint8)[page, :, place] = codes.contiguous().view(torch.uint8)
        if scales is not None:
            scales[page, :, place] = scale


def _gathered(cache, scales, page, place, fmt):
    """Rows of pages and places of any shape, then kv heads of d elements."""
    x = _unpacked(cache.view(torch.uint8)[page, :, place].view(cache.dtype), fmt)
    return x if scales is None else x * scales[page, :, place].float()[..., None]


def _read_plain(s):
    c = s["case"]
    slots = s["slots"].clamp(min=0).long()
    page, place = slots // c["page"], slots % c["page"]
    there = (s["slots"] >= 0)[:, None, None]
    t = _TYPES[c["x"]]
    rows = [_gathered(cache, scales, page, place, c["format"])
            for cache, scales in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"]))]
    return {n: torch.where(there, x, 0.0).to(t) for n, x in zip("kv", rows)}


def _attend_plain(s):
    c = s["case"]
    rows, heads, kv, d = c["rows"], c["heads"], c["kv"], c["d"]
    at = torch.arange(c["length"], device="cuda")
    page, place = s["tables"].long()[:, at // c["page"]], (at % c["page"])[None, :]
    lens = s["lens"][:, None]
    first = (lens - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(lens)
    seen = (at < lens) & (at >= first) & (page >= 0)
    page = page.clamp(min=0)
    k = _gathered(s["k_cache"], s["k_scales"], page, place, c["format"])
    q = s["q"].float().reshape(rows, kv, heads // kv, d).transpose(2, 3).contiguous()
    w = (k.transpose(1, 2).contiguous() @ q) * (1.0 / math.sqrt(d))     # [rows, kv, tokens, share]
    del k
    w = torch.where(seen[:, None, :, None], w, -math.inf).transpose(2, 3).contiguous()
    top = w.amax(3, keepdim=True)
    w = torch.exp(w - torch.where(top > -math.inf, top, 0.0))
    total = w.sum(3, keepdim=True)
    v = _gathered(s["v_cache"], s["v_scales"], page, place, c["format"])
    v = torch.where(seen[:, :, None, None], v, 0.0).transpose(1, 2).contiguous()
    y = (w @ v) / torch.where(total > 0, total, 1.0)
    out = {"y": y.reshape(rows, heads, d).to(_TYPES[c["y"]])}
    if c["lse"]:
        out["lse"] = (top + torch.log(total)).reshape(rows, heads)
    return out


def _state_of(s):
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scales", "v_scales") if s[n] is not None}


def run(state):
    s = state
    c = s["case"]
    kind = c["kind"]
    if not own:
        if kind in ("write", "store", "step"):
            _write_plain(s)
        if kind == "write":
            return _state_of(s)
        if kind == "store":
            return dict(_read_plain(s), k_scales=s["k_scales"], v_scales=s["v_scales"])
        if kind == "read":
            return _read_plain(s)
        out = _attend_plain(s)
        return dict(out, **_state_of(s)) if kind == "step" else out
    import learnable_butterfly_rotation_amd as B
    cache = (s["k_cache"], s["v_cache"])
    scales = {"k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    if kind in ("write", "store", "step"):
        B.bfly_cache_write(s["k"], s["v"], s["slots"], *cache, **scales)
    if kind == "write":
        return _state_of(s)
    if kind == "store":
        B.bfly_cache_read(*cache, s["slots"], s["k_out"], s["v_out"], **scales)
        return {"k": s["k_out"], "v": s["v_out"], **scales}
    if kind == "read":
        B.bfly_cache_read(*cache, s["slots"], s["k"], s["v"], **scales)
        return {"k": s["k"], "v": s["v"]}
    B.bfly_cache_attention(s["q"], *cache, s["tables"], s["lens"], s["y"], max_len=c["length"],
                           window=c["window"], lse=s["lse"], workspace=s["workspace"], **scales)
    out = {"y": s["y"]}
    if c["lse"]:
        out["lse"] = s["lse"]
    return dict(out, **_state_of(s)) if kind == "step" else out


# ---------------------------------------------------------------------------
# the definitions in 64 bits, and the work that a pass cannot do without
# ---------------------------------------------------------------------------

def _numbers(cache, fmt):
    """The numbers that pages stand for, before their scales."""
    if fmt != "int4":
        return cache.to(torch.float64)
    out = torch.empty((*cache.shape[:-1], 2 * cache.shape[-1]), dtype=torch.float64, device="cuda")
    for half in (0, 1):
        nibble = (cache.to(torch.int32) >> (4 * half)) % 16
        out[..., half::2] = torch.where(nibble < 8, nibble, nibble - 16).double()
    return out


def _definition(x, fmt):
    """(what a row is held as, its scale as it is held, the scale unrounded)."""
    x = x.to(torch.float64)
    if fmt == "bf16":
        return x, None, None
    top = _TOP[fmt]
    raw = torch.linalg.vector_norm(x, ord=math.inf, dim=-1) / top
    held = torch.clamp(raw, max=65504.0).half().double()
    ratio = x / torch.where(held > 0, held, math.inf)[..., None]
    if fmt == "e4m3":
        return ratio.clamp(-top, top).to(torch.float8_e4m3fn).double(), held, raw
    return ratio.clamp(-top, top).round(), held, raw


def _written(s, name):
    """The cache after a write, as numbers, with its scales."""
    c = s["case"]
    whole = _numbers(s[name + "_cache"], c["format"])
    scales = None if s[name + "_scales"] is None else s[name + "_scales"].double()
    exact_scales = None if scales is None else scales.clone()
    rows = [t for t, slot in enumerate(s["slots"].tolist()) if slot >= 0]
    slots = s["slots"][rows].long()
    where = (torch.div(slots, c["page"], rounding_mode="floor"), slice(None),
             torch.remainder(slots, c["page"]))
    q, held, raw = _definition(s[name][rows], c["format"])
    whole[where] = q
    if scales is not None:
        scales[where], exact_scales[where] = held, raw
    return whole, scales, exact_scales


def exact(case, seed):
    s = prepare(case, seed)
    kind, fmt, size = case["kind"], case["format"], case["page"]
    out = {}
    if kind in ("write", "store", "step"):
        held = {}
        for n in "kv":
            whole, scales, raw = _written(s, n)
            held[n] = (whole, scales)
            if kind != "store":
                out[n + "_cache"] = None if fmt in ("int8", "int4") else whole
            if scales is not None:
                out[n + "_scales"] = raw
    else:
        held = {n: (_numbers(s[n + "_cache"], fmt),
                    None if s[n + "_scales"] is None else s[n + "_scales"].double()) for n in "kv"}
    if kind == "write":
        return out
    # pages of numbers, scales applied: [pages, kv, page, d]
    pool = {n: x if sc is None else x * sc.unsqueeze(3) for n, (x, sc) in held.items()}
    if kind in ("read", "store"):
        for n in "kv":
            flat = pool[n].permute(0, 2, 1, 3).reshape(-1, case["kv"], case["d"])
            out[n] = flat[s["slots"].clamp(min=0).long()]
            out[n][s["slots"] < 0] = 0.0
        return out
    rows, heads, kv, d = (case[n] for n in ("rows", "heads", "kv", "d"))
    y = torch.zeros((rows, heads, d), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64, device="cuda")
    for r, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        start = max(0, n - case["window"]) if case["window"] else 0
        ids = s["tables"][r, : -(-n // size)].long()
        for h in range(kv):
            k = pool["k"][ids, h].reshape(-1, d)[start:n]
            v = pool["v"][ids, h].reshape(-1, d)[start:n]
            mine = slice(h * heads // kv, (h + 1) * heads // kv)
            score = s["q"][r, mine].double() @ k.T.contiguous() / d ** 0.5
            y[r, mine] = torch.softmax(score, 1) @ v
            lse[r, mine] = torch.logsumexp(score, 1)
    out["y"] = y
    if case["lse"]:
        out["lse"] = lse
    return out


def work(case):
    size = {_BF16: 2, _F32: 4}
    fmt, d, kv = case["format"], case["d"], case["kv"]
    row = d * _ELEMENT[fmt] + (0 if fmt == "bf16" else 2)     # a head's key or value, its scale
    if case["kind"] in ("attend", "step"):
        lens = _lengths(case)
        if case["window"]:
            lens = [min(n, case["window"]) for n in lens]
        tokens, heads, rows = sum(lens), case["heads"], case["rows"]
        b = 2 * tokens * kv * row + sum(4 * -(-n // case["page"]) for n in lens) + 4 * rows
        b += rows * heads * (d * (size[case["q"]] + size[case["y"]]) + (4 if case["lse"] else 0))
        f = 4 * tokens * heads * d
        if case["kind"] == "step":
            b += 2 * rows * kv * (2 * d + row) + 4 * rows
            f += 6 * rows * kv * d
        return {"bytes": b, "flops": f}
    n = case["tokens"]
    moved = n * kv * (row + d * size[case["x"]]) * 2 + 4 * n
    if case["kind"] == "store":
        moved += n * kv * (row + d * size[case["x"]]) * 2
    return {"bytes": moved, "flops": 4 * n * kv * d * (1 if case["kind"] == "read" else 2)}
