"""The operators around a quantized layer, as they are measured: the norm in
front of it with its gradient, the low-rank adapters beside its product and
the clipping of the gradients that its training produces.

`run` computes one pass through one operator: with `own` false in plain torch
operations (fp32 arithmetic whatever the inputs' type; fp64 for the sums whose
result decides roundings next to a border), with `own` true through
learnable_butterfly_rotation_amd.  `exact` gives the same outputs from the
definitions in fp64.  The cases of one operator differ in `kind`:

* norm: h = x + residual (rounded to x's type), y = h / sqrt(mean(h^2) + eps)
  * weight; y itself and/or y in 8 bits (int8 or e4m3) with an fp16 scale per
  group or per row;
* norm_grad: dx = dh + (g - h * mean(g * h) * rstd^2) * rstd with
  g = dy * weight, dweight = sum over rows of dy * h * rstd;
* lora: y = base + scaling[id] * lora_b[id] (lora_a[id] x) for every row, id
  the row's adapter or -1 for none;
* clip: the 2-norm over all tensors, and every tensor times
  min(1, max_norm / norm).
"""
import math

import torch

own = False

_BF16, _F32 = "bf16", "f32"
_TYPES = {_BF16: torch.bfloat16, _F32: torch.float32}
_EPS = 1e-5


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of a decode step: the residual stream's addition, the norm
        # and one scale for the row; latency is all that counts
        {"name": "norm_token_int8", "kind": "norm", "rows": 1, "n": 4096, "x": _BF16,
         "residual": True, "y": "", "format": "int8", "group": 4096},
        # a prompt of 8192 tokens with the group size of the framework's other
        # quantized rows
        {"name": "norm_prompt_int8", "kind": "norm", "rows": 8192, "n": 4096, "x": _BF16,
         "residual": True, "y": "", "format": "int8", "group": 128},
        # a ragged batch that keeps the bf16 rows beside the e4m3 ones (one
        # projection reads 16 bits, the others 8)
        {"name": "norm_batch_e4m3", "kind": "norm", "rows": 777, "n": 5120, "x": _BF16,
         "residual": True, "y": _BF16, "format": "e4m3", "group": 5120},
        # calibration rows in fp32, of a width that no vector load divides
        {"name": "norm_odd_f32", "kind": "norm", "rows": 4099, "n": 1023, "x": _F32,
         "residual": False, "y": _F32, "format": "", "group": 0},
        # the backward of the prompt's norm in bf16, the residual stream's
        # gradient added
        {"name": "norm_grad_bf16", "kind": "norm_grad", "rows": 8192, "n": 4096, "x": _BF16,
         "g": _BF16, "dh": True},
        # fp32 calibration rows at the Kronecker width 5 * 1024
        {"name": "norm_grad_f32", "kind": "norm_grad", "rows": 16384, "n": 5120, "x": _F32,
         "g": _F32, "dh": False},
        # a decode step of 16 requests over 8 adapters
        {"name": "lora_decode", "kind": "lora", "rows": 16, "k": 4096, "n_out": 4096, "rank": 16,
         "adapters": 8, "mixed": True, "base": _BF16, "y": _BF16},
        # a large decode batch at the down projection, 32 adapters in use
        {"name": "lora_batch", "kind": "lora", "rows": 257, "k": 11008, "n_out": 4096, "rank": 64,
         "adapters": 32, "mixed": True, "base": _BF16, "y": _BF16},
        # packed prompts of 6 requests at the up projection, added to the
        # product's fp32 rows
        {"name": "lora_prompts", "kind": "lora", "rows": 8192, "k": 4096, "n_out": 11008,
         "rank": 32, "adapters": 6, "mixed": False, "base": _F32, "y": _BF16},
        # the angle gradients of 24 layers of four rotations of n = 4096
        {"name": "clip_angles", "kind": "clip", "count": 96, "numel": 24576, "ragged": False,
         "g": _F32, "max_norm": 1.0},
        # norm weights, angles and small matrices of odd sizes, below the limit
        {"name": "clip_ragged", "kind": "clip", "count": 300, "numel": 180000, "ragged": True,
         "g": _BF16, "max_norm": 1e4},
        # the weight gradients of 16 layers' 4096 x 11008 matrices
        {"name": "clip_weights", "kind": "clip", "count": 16, "numel": 4096 * 11008,
         "ragged": False, "g": _F32, "max_norm": 1.0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng):
    """A row's length: mostly what the framework rotates, else any."""
    return rng.choice([256, 512, 1024, 2048, 4096, 5120, 8192, 11008, rng.randrange(64, 1024) * 8,
                       rng.randrange(8, 512) * 16, rng.randrange(65, 8192)])


def draw(rng):
    kind = rng.choice(["norm", "norm_grad", "lora", "clip"])
    if kind in ("norm", "norm_grad"):
        n = _width(rng)
        rows = _log_int(rng, 1, min(16384, (1 << 26) // n))
        x = rng.choice([_BF16, _F32])
        if kind == "norm_grad":
            return {"kind": kind, "rows": rows, "n": n, "x": x, "g": rng.choice([_BF16, _F32]),
                    "dh": rng.random() < 0.5}
        fmt = rng.choice(["", "int8", "e4m3"])
        groups = [n] + [g for g in (8, 16, 32, 64, 128, 256, 512) if n % g == 0]
        if fmt == "e4m3":
            rows = max(1, min(rows, 4000000 // n))
        return {"kind": kind, "rows": rows, "n": n, "x": x, "residual": rng.random() < 0.6,
                "y": rng.choice([_BF16, _F32]) if not fmt else rng.choice(["", _BF16, _F32]),
                "format": fmt, "group": rng.choice(groups) if fmt else 0}
    if kind == "lora":
        mixed = rng.random() < 0.5
        rows = _log_int(rng, 1, 512 if mixed else 8192)
        return {"kind": kind, "rows": rows, "k": rng.choice([1024, 4096, 5120, 11008,
                                                             rng.randrange(8, 1024) * 8]),
                "n_out": rng.choice([1024, 4096, 5120, 11008, rng.randrange(8, 1024) * 8]),
                "rank": rng.choice([8, 16, 16, 32, 64, 64, 128, 24, 40]),
                "adapters": _log_int(rng, 1, 48), "mixed": mixed,
                "base": rng.choice([_BF16, _F32, ""]), "y": rng.choice([_BF16, _F32])}
    numel = _log_int(rng, 100, 1 << 24)
    return {"kind": kind, "count": _log_int(rng, 1, min(400, (1 << 28) // numel)), "numel": numel,
            "ragged": rng.random() < 0.7, "g": rng.choice([_BF16, _F32]),
            "max_norm": rng.choice([1.0, 0.1, 1e4])}


# ---------------------------------------------------------------------------
# what a program has in hand before the call
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _activations(g, rows, n, dtype):
    """N(0, 1) rows with 0.1 % of the channels 50 times as large."""
    x = torch.randn((rows, n), generator=g, device="cuda", dtype=torch.float32)
    cols = torch.randperm(n, generator=g, device="cuda")[: int(round(0.001 * n))]
    x[:, cols] *= 50.0
    return x.to(dtype)


def _sizes(case):
    """Elements of every tensor of a clip case."""
    count, numel = case["count"], case["numel"]
    if not case["ragged"]:
        return [numel] * count
    g = torch.Generator().manual_seed(1000 * count + numel)
    u = torch.rand(count, generator=g, dtype=torch.float64)
    sizes = (u * numel).long().tolist()
    sizes[0] = numel
    return sizes


def prepare(case, seed):
    g = _generator(seed)
    kind = case["kind"]
    s = {"case": case}
    if kind in ("norm", "norm_grad"):
        rows, n, dt = case["rows"], case["n"], _TYPES[case["x"]]
        s["weight"] = 1.0 + 0.1 * _randn(g, (n,))
        if kind == "norm":
            s["x"] = _activations(g, rows, n, dt)
            s["residual"] = _activations(g, rows, n, dt) if case["residual"] else None
            s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
            s["y"] = torch.empty((rows, n), dtype=_TYPES[case["y"]], device="cuda") \
                if case["y"] else None
            s["rstd"] = torch.empty(rows, device="cuda")
            s["codes"] = s["scales"] = None
            if case["format"]:
                t = torch.int8 if case["format"] == "int8" else torch.float8_e4m3fn
                s["codes"] = torch.empty((rows, n), dtype=t, device="cuda")
                s["scales"] = torch.empty((rows, n // case["group"]), dtype=torch.float16,
                                          device="cuda")
        else:
            gt = _TYPES[case["g"]]
            s["h"] = _activations(g, rows, n, dt)
            s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + _EPS).float()
            s["dy"] = _randn(g, (rows, n), gt)
            s["dh"] = _randn(g, (rows, n), gt) if case["dh"] else None
            s["dx"] = torch.empty((rows, n), dtype=gt, device="cuda")
            s["dweight"] = torch.empty(n, device="cuda")
            if own:  # scratch that only the framework's call takes
                import learnable_butterfly_rotation_amd as B
                s["workspace"] = torch.empty(B.bfly_rmsnorm_backward_workspace_bytes(rows, n),
                                             dtype=torch.uint8, device="cuda")
    elif kind == "lora":
        rows, k, n_out, r, num = (case[v] for v in ("rows", "k", "n_out", "rank", "adapters"))
        s["x"] = _activations(g, rows, k, torch.bfloat16)
        ids = torch.randint(-1, num, (rows,), generator=g, device="cuda", dtype=torch.int32)
        if not case["mixed"]:  # packed prompts: runs of rows of one request, of uneven lengths
            cuts = torch.randint(0, rows, (num,), generator=g, device="cuda")
            ids = (torch.arange(rows, device="cuda")[:, None] >= cuts[None, :]).sum(1) - 1
            ids = ids.to(torch.int32)
        s["ids"] = ids
        s["lora_a"] = _randn(g, (num, r, k), torch.bfloat16, 1.0 / math.sqrt(k))
        s["lora_b"] = _randn(g, (num, n_out, r), torch.bfloat16, 0.05)
        s["scaling"] = 0.5 + 1.5 * torch.rand(num, generator=g, device="cuda")
        s["base"] = _randn(g, (rows, n_out), _TYPES[case["base"]]) if case["base"] else None
        s["y"] = torch.empty((rows, n_out), dtype=_TYPES[case["y"]], device="cuda")
        if own:
            import learnable_butterfly_rotation_amd as B
            s["workspace"] = torch.empty(
                max(1, B.bfly_lora_matmul_workspace_bytes(rows, n_out, k, r)), dtype=torch.uint8,
                device="cuda")
    else:
        sizes, gt = _sizes(case), _TYPES[case["g"]]
        total = sum(sizes)
        s["flat"] = _randn(g, (total,), gt, 3e-3)
        s["out"] = torch.empty_like(s["flat"])
        s["grads"], s["outs"] = list(s["flat"].split(sizes)), list(s["out"].split(sizes))
        s["norm"] = torch.empty(2, device="cuda")
        if own:
            import learnable_butterfly_rotation_amd as B
            s["workspace"] = torch.empty(B.bfly_grad_clip_workspace_bytes(len(sizes)),
                                         dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _norm_plain(s):
    c = s["case"]
    out = {}
    if s["residual"] is not None:
        out["h"] = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
        h = out["h"].float()
    else:
        h = s["x"].float()
    # the mean square in fp64: a scale or a code next to a rounding border
    # turns on the last bit of y
    rstd = (1.0 / torch.sqrt(h.double().square().mean(1) + float(torch.tensor(_EPS)))).float()
    out["rstd"] = rstd
    y = h * rstd[:, None] * s["weight"]
    if c["y"]:
        out["y"] = y.to(_TYPES[c["y"]])
    if c["format"]:
        top = 127.0 if c["format"] == "int8" else 448.0
        v = y.reshape(c["rows"], -1, c["group"])
        scale = (v.abs().amax(2) / top).clamp(max=65504.0).to(torch.float16)
        d = scale.float()[:, :, None]
        q = torch.where(d > 0, v / d, torch.zeros_like(v)).clamp(-top, top)
        q = q.reshape(c["rows"], c["n"])
        out["codes"] = torch.round(q).to(torch.int8) if c["format"] == "int8" \
            else q.to(torch.float8_e4m3fn)
        out["scales"] = scale
    return out


def _norm_grad_plain(s):
    h, dy, r = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    g = dy * s["weight"]
    xhat = h * r
    dx = (g - xhat * (g * xhat).mean(1, keepdim=True)) * r
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * xhat).double().sum(0).float()}


def _lora_plain(s):
    c = s["case"]
    num, r = c["adapters"], c["rank"]
    # every row against every adapter, then all but the row's own dropped
    t = (s["x"].float() @ s["lora_a"].float().reshape(num * r, -1).T).reshape(-1, num, r)
    mine = s["ids"][:, None] == torch.arange(num, device="cuda", dtype=torch.int32)
    t = torch.where(mine[:, :, None], t * s["scaling"][None, :, None], torch.zeros_like(t))
    y = t.reshape(-1, num * r) @ s["lora_b"].float().permute(0, 2, 1).reshape(num * r, -1)
    if s["base"] is not None:
        y = s["base"].float() + y
    return y.to(_TYPES[c["y"]])


def _clip_plain(s):
    sq = torch.stack([g.double().square().sum() for g in s["grads"]]).sum()
    norm = torch.sqrt(sq)
    coef = torch.clamp(s["case"]["max_norm"] / norm, max=1.0).float()
    outs = [(g.float() * coef).to(g.dtype) for g in s["grads"]]
    return {"norm": torch.stack([norm.float(), coef]), "out": torch.cat(outs)}


def run(state):
    s = state
    c = s["case"]
    kind = c["kind"]
    if not own:
        return {"norm": _norm_plain, "norm_grad": _norm_grad_plain, "lora": _lora_plain,
                "clip": _clip_plain}[kind](s)
    import learnable_butterfly_rotation_amd as B
    if kind == "norm":
        B.bfly_rmsnorm(s["x"], s["weight"], _EPS, y=s["y"], codes=s["codes"], scales=s["scales"],
                       residual=s["residual"], h=s["h"], rstd=s["rstd"],
                       format=B.BFLY_Q8_E4M3 if c["format"] == "e4m3" else B.BFLY_Q8_INT8,
                       group=c["group"])
        return {k: s[k] for k in ("h", "rstd", "y", "codes", "scales") if s[k] is not None}
    if kind == "norm_grad":
        B.bfly_rmsnorm_backward(s["h"], s["weight"], s["rstd"], s["dy"], s["dx"],
                                dweight=s["dweight"], dh=s["dh"], workspace=s["workspace"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if kind == "lora":
        B.bfly_lora_matmul(s["x"], s["ids"], s["lora_a"], s["lora_b"], s["scaling"], s["y"],
                           s["workspace"], base=s["base"])
        return s["y"]
    B.bfly_grad_clip(s["grads"], c["max_norm"], s["norm"], s["workspace"], outs=s["outs"])
    return {"norm": s["norm"], "out": s["out"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, and the work that a pass cannot do without
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        x = s["x"].double()
        out = {}
        if s["residual"] is not None:
            x = (x + s["residual"].double()).to(s["x"].dtype).double()
            out["h"] = x
        ms = (x * x).sum(1, keepdim=True) / case["n"]
        r = (ms + float(torch.tensor(_EPS))) ** -0.5
        out["rstd"] = r[:, 0]
        y = x * r * s["weight"].double()
        if case["y"]:
            out["y"] = y
        if case["format"]:
            top = {"int8": 127.0, "e4m3": 448.0}[case["format"]]
            group = y.view(case["rows"], case["n"] // case["group"], case["group"])
            scale = group.abs().max(dim=2).values / top
            held = scale.half().double().clamp(min=2.0 ** -24)
            q = (group / held[..., None]).view(case["rows"], case["n"])
            out["codes"] = None if case["format"] == "int8" \
                else q.clamp(-top, top).float().to(torch.float8_e4m3fn).double()
            out["scales"] = scale
        return out
    if kind == "norm_grad":
        h, dy, w, r = (s[v].double() for v in ("h", "dy", "weight", "rstd"))
        dot = torch.einsum("ij,j,ij->i", dy, w, h)
        dx = torch.outer(r, w) * dy - h * (dot * r ** 3 / case["n"])[:, None]
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dweight": torch.mv((dy * h).T, r)}
    if kind == "lora":
        y = s["base"].double() if s["base"] is not None else \
            torch.zeros((case["rows"], case["n_out"]), dtype=torch.float64, device="cuda")
        for a in range(case["adapters"]):
            at = torch.nonzero(s["ids"] == a)[:, 0]
            if len(at):
                t = s["x"][at].double() @ s["lora_a"][a].double().T.contiguous()
                y[at] += s["scaling"][a].double() * (t @ s["lora_b"][a].double().T.contiguous())
        return y
    flat = s["flat"].double()
    norm = torch.linalg.vector_norm(flat)
    coef = min(1.0, case["max_norm"] / float(norm))
    return {"norm": torch.stack([norm, norm.new_tensor(coef)]), "out": flat.mul_(coef)}


def work(case):
    size = {_BF16: 2, _F32: 4, "": 0}
    kind = case["kind"]
    if kind in ("norm", "norm_grad"):
        rows, n = case["rows"], case["n"]
        e = rows * n
        if kind == "norm":
            b = e * size[case["x"]] * (3 if case["residual"] else 1) + e * size[case["y"]]
            b += (e + 2 * e // case["group"]) if case["format"] else 0
            return {"bytes": b + 4 * rows + 4 * n, "flops": 6 * e}
        b = e * size[case["x"]] + e * size[case["g"]] * (3 if case["dh"] else 2)
        return {"bytes": b + 4 * rows + 8 * n, "flops": 10 * e}
    if kind == "lora":
        rows, k, n_out, r = case["rows"], case["k"], case["n_out"], case["rank"]
        used = min(case["adapters"], rows)
        return {"bytes": 2 * rows * k + 4 * rows + 2 * used * r * (k + n_out) +
                rows * n_out * (size[case["base"]] + size[case["y"]]),
                "flops": 2 * rows * r * (k + n_out)}
    total = sum(_sizes(case))
    return {"bytes": 2 * total * size[case["g"]] + 8, "flops": 3 * total}
