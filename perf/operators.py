"""Cases of the 8-bit and expert-grouped operators: real sizes, their inputs, their plain forms and
their definitions in 64 bits.

Five entry points are measured:

* ``coco_allreduce_rmsnorm``: the sum over ranks of a row-parallel product's partials, the residual's
  addition and the root-mean-square norm, with the normalised rows in 16/32 bits or in e4m3 with one
  scale per row and 128 columns;
* ``coco_allreduce_rmsnorm_backward``: its gradient (rank-partial gradients summed in the same pass);
* ``coco_quantize_fp8``: e4m3 values and scales of activations (1 x 128) or weights (128 x 128);
* ``coco_einsum_fp8``: the product of e4m3 operands with such scales;
* ``coco_grouped_einsum``: products grouped by expert with ragged sizes, their input gradients (the
  transposed form) and their weight gradients.

With ``own`` false ``run`` computes a case in elementary torch operations in 32 bits, rounded once at
the end; with ``own`` true it calls the framework.
"""

import torch

own = False

BLOCK = 128  # columns (and weight rows) that share a scale
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # the smallest block maximum a scale is made from
EPS = 1e-5

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}


def listed():
    return [
        # One decoded token on eight ranks: latency of the layer's tail, ready for an 8-bit product.
        {"name": "norm one token", "op": "norm", "dtype": "bf16", "ranks": 8, "rows": 1, "cols": 4096, "out": "fp8",
         "copies": 1},
        # The Megatron tail at its full size (8 x 1024 tokens of 4096, fp16, 8 ranks), every rank with its copy.
        {"name": "norm megatron", "op": "norm", "dtype": "f16", "ranks": 8, "rows": 8192, "cols": 4096, "out": "fp8",
         "copies": 8},
        # Backward of a ragged microbatch, two ranks.
        {"name": "norm grad ragged", "op": "norm_grad", "dtype": "bf16", "ranks": 2, "rows": 777, "cols": 8192},
        # Backward of the Megatron tail at its full size.
        {"name": "norm grad megatron", "op": "norm_grad", "dtype": "f16", "ranks": 8, "rows": 8192, "cols": 4096},
        # The MLP's activations of a decoding batch, between its two products.
        {"name": "quantise decode", "op": "quantise", "dtype": "bf16", "ranks": 1, "rows": 33, "cols": 32768,
         "block": 1},
        # A layer's weight (the 2-D mesh MLP's W1) brought to 8 bits.
        {"name": "quantise weight", "op": "quantise", "dtype": "bf16", "ranks": 1, "rows": 8192, "cols": 32768,
         "block": 128},
        # One decoded token through a square projection: the weight's bytes are all there is.
        {"name": "product one token", "op": "product", "ranks": 1, "m": 1, "k": 4096, "n": 4096, "form": "nk",
         "out": "bf16"},
        # A ragged prefill chunk, row-parallel over eight ranks, sizes that end inside blocks.
        {"name": "product ragged", "op": "product", "ranks": 8, "m": 333, "k": 528, "n": 4112, "form": "kn",
         "out": "bf16"},
        # A training or prefill product.
        {"name": "product large", "op": "product", "ranks": 1, "m": 8192, "k": 8192, "n": 8192, "form": "kn",
         "out": "bf16"},
        # Sixteen decoded tokens, two experts each, of 64: a few rows an expert, some with none.
        {"name": "experts decode", "op": "grouped", "dtype": "fp8", "rows": 32, "experts": 64, "k": 4096, "n": 2048,
         "form": "nk", "skew": 1.0},
        # Training, 8192 tokens with two experts each of 32, unevenly spread.
        {"name": "experts forward", "op": "grouped", "dtype": "bf16", "rows": 16384, "experts": 32, "k": 4096,
         "n": 2048, "form": "kn", "skew": 1.0},
        # The weight gradient of the same.
        {"name": "experts weight grad", "op": "grouped", "dtype": "bf16", "rows": 16384, "experts": 32, "k": 4096,
         "n": 2048, "form": "grad", "skew": 1.0},
    ]


def _log(rng, low, high):
    """A whole number spread evenly over the logarithm of [low, high]."""
    return max(low, min(high, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quantise", "product", "product", "grouped", "grouped"])
    if op in ("norm", "norm_grad"):
        ranks = rng.choice([1, 2, 3, 4, 8])
        cols = 16 * _log(rng, 8, 1024)
        rows = _log(rng, 1, max(1, min(16384, 8192 * 4096 * 8 // (ranks * cols))))
        case = {"op": op, "dtype": rng.choice(["bf16", "f16"]), "ranks": ranks, "rows": rows, "cols": cols}
        if op == "norm":
            case["out"] = rng.choice(["fp8", "fp8", "same"])
            case["copies"] = rng.choice([1, ranks])
        return case
    if op == "quantise":
        cols = 16 * _log(rng, 8, 2048)
        return {"op": op, "dtype": rng.choice(["bf16", "f16", "f32"]), "ranks": rng.choice([1, 2]),
                "rows": _log(rng, 1, min(16384, 8192 * 32768 // (2 * cols))), "cols": cols,
                "block": rng.choice([1, 1, 128])}
    if op == "product":
        ranks = rng.choice([1, 1, 2, 8])
        k, n = 16 * _log(rng, 16, 512), 16 * _log(rng, 16, 512)
        return {"op": op, "ranks": ranks, "m": _log(rng, 1, max(1, min(8192, 8192 ** 3 // (ranks * k * n)))), "k": k,
                "n": n, "form": rng.choice(["kn", "nk"]), "out": rng.choice(["bf16", "bf16", "f16"])}
    form = rng.choice(["kn", "nk", "grad"])
    return {"op": op, "dtype": rng.choice(["bf16", "f16"] if form == "grad" else ["fp8", "fp8", "bf16", "f16"]),
            "rows": _log(rng, 1, 16384), "experts": rng.choice([1, 5, 8, 32, 64]), "k": 16 * _log(rng, 16, 256),
            "n": 16 * _log(rng, 16, 128), "form": form, "skew": rng.choice([0.0, 1.0, 2.0])}


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _activations(g, shape, dtype, std=1.0):
    """Rows of a transformer's stream: normal values, one column in 64 some ten times larger."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)
    x[..., ::64] *= 10.0
    return x.to(dtype)


def _held_in_8_bits(x, block_rows):
    """e4m3 values and scales of the last two dimensions of x, in blocks of block_rows x 128."""
    rows, cols = x.shape[-2:]
    up = torch.nn.functional.pad(x.float(), (0, -cols % BLOCK, 0, -rows % block_rows))
    tiles = up.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, block_rows))  # [.., R, br, C, 128]
    scales = tiles.abs().amax((-3, -1)).clamp_min(AMAX_FLOOR) / E4M3_MAX
    q = (tiles / scales[..., :, None, :, None]).flatten(-4, -3).flatten(-2, -1)[..., :rows, :cols]
    return q.to(torch.float8_e4m3fn).contiguous(), scales.contiguous()


def _counts(seed, rows, experts, skew):
    """Rows of every expert: shares like 1 / rank^skew in a random order, whole numbers that sum to `rows`."""
    g = torch.Generator().manual_seed(seed)
    share = (torch.randperm(experts, generator=g) + 1).double().pow(-skew)
    pick = torch.multinomial(share, rows, replacement=True, generator=g)
    return torch.bincount(pick, minlength=experts).tolist()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        ranks, rows, cols, dt = case["ranks"], case["rows"], case["cols"], DTYPES[case["dtype"]]
        s["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(dt)
    if op == "norm":
        s["partials"] = _activations(g, (ranks, rows, cols), dt, ranks ** -0.5)
        s["residual"] = _activations(g, (rows, cols), dt)
        out = DTYPES["fp8"] if case["out"] == "fp8" else dt
        n = case["copies"]
        s["hidden"] = [torch.empty(rows, cols, dtype=dt, device="cuda") for _ in range(n)]
        s["normed"] = [torch.empty(rows, cols, dtype=out, device="cuda") for _ in range(n)]
        s["scales"] = [torch.empty(rows, _blocks(cols), device="cuda") for _ in range(n)] \
            if case["out"] == "fp8" else None
        s["rstd"] = torch.empty(rows, device="cuda")
    elif op == "norm_grad":
        s["dnormed"] = (torch.randn(ranks, rows, cols, generator=g, device="cuda") * ranks ** -0.5).to(dt)
        s["dhidden"] = torch.randn(rows, cols, generator=g, device="cuda").to(dt)
        s["hidden"] = _activations(g, (rows, cols), dt)
        s["rstd"] = (s["hidden"].float().square().mean(-1) + EPS).rsqrt()
        s["dx"] = torch.empty(rows, cols, dtype=dt, device="cuda")
        s["dweight"] = torch.empty(cols, device="cuda")
    elif op == "quantise":
        ranks, rows, cols = case["ranks"], case["rows"], case["cols"]
        s["x"] = _activations(g, (ranks, rows, cols), DTYPES[case["dtype"]])
        s["q"] = torch.empty(ranks, rows, cols, dtype=DTYPES["fp8"], device="cuda")
        s["scales"] = torch.empty(ranks, -(-rows // case["block"]), _blocks(cols), device="cuda")
    elif op == "product":
        ranks, m, k, n = case["ranks"], case["m"], case["k"], case["n"]
        s["lhs"], s["lhs_scales"] = _held_in_8_bits(_activations(g, (ranks, m, k), torch.float32), 1)
        shape = (ranks, k, n) if case["form"] == "kn" else (ranks, n, k)
        s["rhs"], s["rhs_scales"] = _held_in_8_bits(
            torch.randn(shape, generator=g, device="cuda") * k ** -0.5, BLOCK)
        s["out"] = torch.empty(ranks, m, n, dtype=DTYPES[case["out"]], device="cuda")
    else:
        rows, experts, k, n, form = case["rows"], case["experts"], case["k"], case["n"], case["form"]
        dt = DTYPES[case["dtype"]]
        s["counts"] = _counts(seed, rows, experts, case["skew"])
        s["offsets"] = torch.tensor([0] + s["counts"]).cumsum(0).to("cuda", torch.int32)
        if form == "grad":
            s["lhs"] = _activations(g, (rows, k), dt)
            s["rhs"] = torch.randn(rows, n, generator=g, device="cuda").to(dt)
            s["out"] = torch.empty(experts, k, n, dtype=dt, device="cuda")
            return s
        lhs = _activations(g, (rows, k), torch.float32)
        rhs = torch.randn((experts, k, n) if form == "kn" else (experts, n, k), generator=g, device="cuda")
        rhs *= k ** -0.5
        if case["dtype"] == "fp8":
            s["lhs"], s["lhs_scales"] = _held_in_8_bits(lhs, 1)
            s["rhs"], s["rhs_scales"] = _held_in_8_bits(rhs, BLOCK)
            s["out"] = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
        else:
            s["lhs"], s["rhs"] = lhs.to(dt), rhs.to(dt)
            s["out"] = torch.empty(rows, n, dtype=dt, device="cuda")
    return s


def run(s):
    return _framework(s) if own else _plain(s)


# ------------------------------------------------------------------------------ the framework's calls


def _framework(s):
    from collective_fusedallreduce_gb300 import coco

    case = s["case"]
    op = case["op"]
    if op == "norm":
        n, copies = case["ranks"], case["copies"]
        spread = (lambda v: v) if copies == n else (lambda v: v * n)  # a copy for every rank, or one for all
        coco.coco_allreduce_rmsnorm(
            coco.local(list(s["partials"])), coco.replicated([s["residual"]] * n), s["weight"], EPS,
            coco.replicated(spread(s["hidden"])), coco.replicated(spread(s["normed"])),
            spread(s["scales"]) if s["scales"] else None, s["rstd"])
        return {"hidden": s["hidden"], "normed": s["normed"], "scales": s["scales"], "rstd": s["rstd"]}
    if op == "norm_grad":
        n, rows, cols = case["ranks"], case["rows"], case["cols"]
        space = torch.empty(coco.coco_allreduce_rmsnorm_backward_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        coco.coco_allreduce_rmsnorm_backward(
            coco.local(list(s["dnormed"])), coco.replicated([s["dhidden"]] * n), coco.replicated([s["hidden"]] * n),
            s["weight"], s["rstd"], coco.replicated([s["dx"]] * n), s["dweight"], space)
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if op == "quantise":
        coco.coco_quantize_fp8(coco.local(list(s["x"])), case["block"], coco.local(list(s["q"])), list(s["scales"]))
        return {"q": s["q"], "scales": s["scales"]}
    if op == "product":
        coco.coco_einsum_fp8("mk,kn->mn" if case["form"] == "kn" else "mk,nk->mn", coco.local(list(s["lhs"])),
                             list(s["lhs_scales"]), coco.local(list(s["rhs"])), list(s["rhs_scales"]),
                             coco.local(list(s["out"])))
        return s["out"]
    spec = {"kn": "tk,ekn->tn", "nk": "tk,enk->tn", "grad": "tk,tn->ekn"}[case["form"]]
    fp8 = case["dtype"] == "fp8"
    coco.coco_grouped_einsum(spec, coco.local([s["lhs"]]), [s["lhs_scales"]] if fp8 else None,
                             coco.local([s["rhs"]]), [s["rhs_scales"]] if fp8 else None, s["offsets"],
                             coco.local([s["out"]]))
    return s["out"]


# ------------------------------------------------------------------------------------- the plain form


def _spread(scales, rows, cols, block_rows):
    """One scale for every value of a [.., rows, cols] operand."""
    up = scales.repeat_interleave(BLOCK, -1)[..., :cols]
    return up if block_rows == 1 else up.repeat_interleave(block_rows, -2)[..., :rows, :]


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        h = s["partials"].float().sum(0) + s["residual"].float()
        rstd = (h.square().mean(-1) + EPS).rsqrt()
        y = h * rstd[:, None] * s["weight"].float()
        dt = s["residual"].dtype
        copies = case["copies"]
        if case["out"] != "fp8":
            q, scales = y.to(dt), None
        else:
            q, scales = _held_in_8_bits(y, 1)
            scales = [scales.clone() for _ in range(copies)]
        return {"hidden": [h.to(dt) for _ in range(copies)], "normed": [q.clone() for _ in range(copies)],
                "scales": scales, "rstd": rstd}
    if op == "norm_grad":
        dy, h, r = s["dnormed"].float().sum(0), s["hidden"].float(), s["rstd"][:, None]
        xhat = h * r
        g = dy * s["weight"].float()
        dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True)) + s["dhidden"].float()
        return {"dx": dx.to(s["hidden"].dtype), "dweight": (dy * xhat).sum(0)}
    if op == "quantise":
        q, scales = _held_in_8_bits(s["x"], case["block"])
        return {"q": q, "scales": scales}
    if op == "product":
        m, k, n = case["m"], case["k"], case["n"]
        lhs = s["lhs"].float() * _spread(s["lhs_scales"], m, k, 1)
        rhs = s["rhs"].float() * _spread(s["rhs_scales"], *s["rhs"].shape[-2:], BLOCK)
        return (lhs @ (rhs if case["form"] == "kn" else rhs.mT)).to(s["out"].dtype)
    rows, k = case["rows"], case["k"]
    lhs, rhs, counts = s["lhs"].float(), s["rhs"].float(), s["counts"]
    if case["form"] == "grad":
        both = zip(lhs.split(counts), rhs.split(counts))
        return torch.stack([a.mT @ b for a, b in both]).to(s["out"].dtype)
    if case["dtype"] == "fp8":
        lhs = lhs * _spread(s["lhs_scales"], rows, k, 1)
        rhs = rhs * _spread(s["rhs_scales"], *s["rhs"].shape[-2:], BLOCK)
    if case["form"] == "nk":
        rhs = rhs.mT
    return torch.cat([a @ b for a, b in zip(lhs.split(counts), rhs)]).to(s["out"].dtype)


# --------------------------------------------------------------------------- the definitions in 64 bits


def _e4m3_of(y, block_rows):
    """(values on the e4m3 grid, scales) of the last two dimensions of y in 64 bits, block by block of columns."""
    *lead, rows, cols = y.shape
    nb, rb = _blocks(cols), -(-rows // block_rows)
    values, scales = torch.empty_like(y), y.new_empty(*lead, rb, nb)
    for b in range(nb):
        part = y[..., b * BLOCK:(b + 1) * BLOCK]
        top = part.abs().amax(-1)
        if block_rows > 1:
            top = torch.stack([t.amax(-1) for t in top.split(block_rows, -1)], -1)
        sc = torch.maximum(top, torch.full_like(top, AMAX_FLOOR)) / E4M3_MAX
        scales[..., b] = sc
        per_row = torch.repeat_interleave(sc, block_rows, -1)[..., :rows] if block_rows > 1 else sc
        v = part / per_row[..., None]
        # e4m3: three fraction bits above 2^-6, steps of 2^-9 below
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))).clamp_min(-6) - 3)
        values[..., b * BLOCK:(b + 1) * BLOCK] = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    return values, scales


def _wide(x, scales=None, block_rows=1):
    """An operand's values in 64 bits."""
    x = x.double()
    if scales is not None:
        for b in range(scales.shape[-1]):
            sc = scales[..., b].double()
            if block_rows > 1:
                sc = torch.repeat_interleave(sc, block_rows, -1)[..., :x.shape[-2]]
            x[..., b * BLOCK:(b + 1) * BLOCK] *= sc[..., None]
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["residual"].double()
        for p in s["partials"]:
            h = h + p.double()
        ms = torch.einsum("rc,rc->r", h, h) / case["cols"]
        rstd = 1.0 / torch.sqrt(ms + EPS)
        y = torch.einsum("rc,r,c->rc", h, rstd, s["weight"].double())
        copies = case["copies"]
        q, scales = _e4m3_of(y, 1) if case["out"] == "fp8" else (y, None)
        return {"hidden": [h] * copies, "normed": [q] * copies,
                "scales": [scales] * copies if scales is not None else None, "rstd": rstd}
    if op == "norm_grad":
        dy = sum(p.double() for p in s["dnormed"])
        h, r, w = s["hidden"].double(), s["rstd"].double(), s["weight"].double()
        # h r w's derivative: w r dy, less h r^3 / C times the row's product of h with w dy
        along = torch.einsum("rc,c,rc->r", dy, w, h)
        dx = dy * w * r[:, None] - h * (r ** 3 * along / case["cols"])[:, None] + s["dhidden"].double()
        return {"dx": dx, "dweight": torch.einsum("rc,rc,r->c", dy, h, r)}
    if op == "quantise":
        q, scales = _e4m3_of(s["x"].double(), case["block"])
        return {"q": q, "scales": scales}
    scaled = op == "product" or case["dtype"] == "fp8"
    lhs = _wide(s["lhs"], s["lhs_scales"] if scaled else None)
    rhs = _wide(s["rhs"], s["rhs_scales"] if scaled else None, BLOCK)
    if op == "product":
        return torch.einsum("rmk,rkn->rmn" if case["form"] == "kn" else "rmk,rnk->rmn", lhs, rhs)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for e, c in enumerate(s["counts"]):
        a = lhs[at:at + c]
        if case["form"] == "grad":
            out[e] = torch.einsum("tk,tn->kn", a, rhs[at:at + c])
        else:
            out[at:at + c] = torch.einsum("tk,kn->tn" if case["form"] == "kn" else "tk,nk->tn", a, rhs[e])
        at += c
    return out


# -------------------------------------------------------------------------------------- the work of a pass


def work(case):
    """Each input read once and each output written once; two operations for a product's multiply and add."""
    op = case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 1}
    if op == "norm":
        v, es = case["rows"] * case["cols"], size[case["dtype"]]
        out = v + 4 * case["rows"] * _blocks(case["cols"]) if case["out"] == "fp8" else v * es
        return {"bytes": v * es * (case["ranks"] + 1) + case["cols"] * es + case["copies"] * (v * es + out)
                + 4 * case["rows"], "flops": v * (case["ranks"] + 6)}
    if op == "norm_grad":
        v, es = case["rows"] * case["cols"], size[case["dtype"]]
        return {"bytes": v * es * (case["ranks"] + 3) + case["cols"] * (es + 4) + 4 * case["rows"],
                "flops": v * (case["ranks"] + 10)}
    if op == "quantise":
        v = case["ranks"] * case["rows"] * case["cols"]
        blocks = case["ranks"] * -(-case["rows"] // case["block"]) * _blocks(case["cols"])
        return {"bytes": v * (size[case["dtype"]] + 1) + 4 * blocks, "flops": 3 * v}
    k, n = case["k"], case["n"]
    if op == "product":
        r, m = case["ranks"], case["m"]
        return {"bytes": r * (m * k + k * n + 2 * m * n + 4 * (m * _blocks(k) + _blocks(k) * _blocks(n))),
                "flops": 2 * r * m * k * n}
    rows, experts, es = case["rows"], case["experts"], size[case["dtype"]]
    flops = 2 * rows * k * n
    if case["form"] == "grad":
        return {"bytes": es * (rows * (k + n) + experts * k * n) + 4 * (experts + 1), "flops": flops}
    # experts that some row goes to; their number is the routing's, so the expected one stands for it
    share = [(i + 1) ** -case["skew"] for i in range(experts)]
    total = sum(share)
    met = sum(1.0 - (1.0 - p / total) ** rows for p in share)
    scales = 4 * (rows * _blocks(k) + met * _blocks(k) * _blocks(n)) if case["dtype"] == "fp8" else 0
    return {"bytes": es * (rows * k + met * k * n) + 2 * rows * n + scales + 4 * (experts + 1), "flops": flops}
