"""Cases of the operators that move tokens to their experts and back, of the layer norm after an AllReduce, and of
clipping by the global gradient norm: real sizes, their inputs, their plain forms and their definitions in 64 bits.

The entry points that are measured:

* ``coco_expert_sort`` and ``coco_expert_dispatch`` (op "dispatch"): the rows of a mixture of experts, sorted by expert;
* ``coco_expert_combine`` (op "combine"): the experts' rows back to their tokens with weights applied, summed over the
  ranks; without weights it is the dispatch's gradient;
* ``coco_expert_combine_backward`` (op "combine_grad"): its gradient, of the rows and of the weights;
* ``coco_allreduce_layernorm`` (op "norm") and ``coco_allreduce_layernorm_backward`` (op "norm_grad"): the sum over
  ranks of a row-parallel product's partials, the residual's addition and the layer norm, and its gradient;
* ``coco_scattered_clip`` (op "clip") and ``coco_scattered_allreduce_clip`` (op "reduce_clip"): gradients in many
  separate tensors, scaled so that their norm is at most a given one, the latter summed over the ranks first.

With ``own`` false ``run`` computes a case in elementary torch operations in 32 bits, rounded once at the end; with
``own`` true it calls the framework.
"""

import torch

own = False

BLOCK = 128  # columns that share a scale of an 8-bit row
E4M3_MAX = 448.0
EPS = 1e-5
GRAD = 1e-3  # a gradient's standard deviation

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
SIZES = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 1}


def listed():
    return [
        # Sixteen decoded tokens, two experts each, of 64, their rows in 8 bits: latency.
        {"name": "dispatch decode", "op": "dispatch", "dtype": "fp8", "tokens": 16, "choices": 2, "experts": 64,
         "cols": 4096, "skew": 1.0, "dropped": 0.0},
        # Training, 8192 tokens with two experts each of 32, unevenly spread; some choices have no place.
        {"name": "dispatch training", "op": "dispatch", "dtype": "bf16", "tokens": 8192, "choices": 2, "experts": 32,
         "cols": 4096, "skew": 1.0, "dropped": 0.02},
        # The way back of the decoded tokens, over eight ranks, into the residual stream.
        {"name": "combine decode", "op": "combine", "dtype": "bf16", "ranks": 8, "tokens": 16, "choices": 2,
         "cols": 4096, "weights": True, "summed": True, "dropped": 0.0},
        # The same for the training tokens.
        {"name": "combine training", "op": "combine", "dtype": "bf16", "ranks": 8, "tokens": 8192, "choices": 2,
         "cols": 4096, "weights": True, "summed": True, "dropped": 0.02},
        # Backward of a ragged microbatch, three experts a token, two ranks.
        {"name": "combine grad ragged", "op": "combine_grad", "dtype": "f16", "ranks": 2, "tokens": 777, "choices": 3,
         "cols": 8192, "dropped": 0.0},
        # Backward of the training tokens.
        {"name": "combine grad training", "op": "combine_grad", "dtype": "bf16", "ranks": 8, "tokens": 8192,
         "choices": 2, "cols": 4096, "dropped": 0.02},
        # One decoded token on eight ranks: latency of the layer's tail.
        {"name": "layer norm one token", "op": "norm", "dtype": "bf16", "ranks": 8, "rows": 1, "cols": 4096,
         "out": "same", "copies": 1},
        # The Megatron tail at its full size (8 x 1024 tokens of 4096, fp16, 8 ranks), every rank with its copy.
        {"name": "layer norm megatron", "op": "norm", "dtype": "f16", "ranks": 8, "rows": 8192, "cols": 4096,
         "out": "same", "copies": 8},
        # Backward of a ragged microbatch, two ranks.
        {"name": "layer norm grad ragged", "op": "norm_grad", "dtype": "bf16", "ranks": 2, "rows": 777, "cols": 8192},
        # Backward of the Megatron tail at its full size.
        {"name": "layer norm grad megatron", "op": "norm_grad", "dtype": "f16", "ranks": 8, "rows": 8192,
         "cols": 4096},
        # The gradients of one transformer layer (16 tensors) to fp32 ones for the optimizer.
        {"name": "clip one layer", "op": "clip", "dtype": "bf16", "out": "f32", "ranks": 1, "layers": 1,
         "hidden": 1024, "words": 0, "share": 0.5},
        # BERT-large's gradients of eight data-parallel ranks, averaged and clipped.
        {"name": "reduce clip bert", "op": "reduce_clip", "dtype": "f16", "out": "f16", "ranks": 8, "layers": 24,
         "hidden": 1024, "words": 30522, "share": 0.5},
    ]


def _log(rng, low, high):
    """A whole number spread evenly over the logarithm of [low, high]."""
    return max(low, min(high, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch", "combine", "combine_grad", "norm", "norm_grad", "clip", "reduce_clip"])
    if op in ("clip", "reduce_clip"):
        hidden = 16 * _log(rng, 2, 64)
        ranks = rng.choice([1, 2, 4]) if op == "clip" else rng.choice([2, 3, 8])
        dtype = rng.choice(["bf16", "f16", "f32"])
        return {"op": op, "dtype": dtype, "out": rng.choice([dtype, "f32"]), "ranks": ranks,
                "layers": _log(rng, 1, max(1, min(24, 24 * 4 * SIZES["f16"] // (ranks * SIZES[dtype])))),
                "hidden": hidden, "words": rng.choice([0, 101, 2049]), "share": rng.choice([0.5, 0.5, 2.0])}
    if op in ("norm", "norm_grad"):
        ranks = rng.choice([1, 2, 3, 4, 8])
        cols = 16 * _log(rng, 8, 1024)
        rows = _log(rng, 1, max(1, min(16384, 8192 * 4096 * 8 // (ranks * cols))))
        case = {"op": op, "dtype": rng.choice(["bf16", "f16", "bf16", "f16", "f32"]), "ranks": ranks, "rows": rows,
                "cols": cols}
        if case["dtype"] == "f32":
            case["rows"] = max(1, rows // 2)
        if op == "norm":
            case["out"] = rng.choice(["fp8", "same", "same"])
            case["copies"] = rng.choice([1, ranks])
        return case
    cols = 16 * _log(rng, 8, 512)
    choices = rng.choice([1, 2, 2, 3, 4, 8])
    ranks = 1 if op == "dispatch" else rng.choice([1, 2, 3, 8])
    case = {"op": op, "dtype": rng.choice(["bf16", "f16"]), "ranks": ranks,
            "tokens": _log(rng, 1, max(1, min(16384, 8192 * 4096 * 2 * 8 // (ranks * choices * cols)))),
            "choices": choices, "cols": cols, "dropped": rng.choice([0.0, 0.0, 0.1])}
    if op == "dispatch":
        del case["ranks"]
        case["dtype"] = rng.choice(["fp8", "bf16", "f16", "f32"])
        case["experts"] = rng.choice([1, 5, 8, 32, 64, 257, 1024])
        case["skew"] = rng.choice([0.0, 1.0, 2.0])
    elif op == "combine":
        case["weights"], case["summed"] = rng.choice([True, True, False]), rng.choice([True, False])
    return case


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _activations(g, shape, dtype, std=1.0):
    """Rows of a transformer's stream: normal values off centre, one column in 64 some ten times larger."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).add_(0.25).mul_(std)
    x[..., ::64] *= 10.0
    return x.to(dtype)


def _held_in_8_bits(x):
    """e4m3 values and scales of rows, a scale per 128 columns."""
    cols = x.shape[-1]
    tiles = torch.nn.functional.pad(x.float(), (0, -cols % BLOCK)).unflatten(-1, (-1, BLOCK))
    scales = tiles.abs().amax(-1).clamp_min(2.0 ** -100) / E4M3_MAX
    q = (tiles / scales[..., None]).flatten(-2)[..., :cols]
    return q.to(torch.float8_e4m3fn).contiguous(), scales.contiguous()


def _routing(g, case, experts, skew):
    """A token's choices [tokens, choices]: experts with shares like 1 / rank^skew, a choice without a place is -1."""
    share = (torch.randperm(experts, generator=g, device="cuda") + 1).double().pow(-skew).float()
    n = case["tokens"] * case["choices"]
    pick = torch.multinomial(share, n, replacement=True, generator=g)
    lost = torch.rand(n, generator=g, device="cuda") < case["dropped"]
    return torch.where(lost, -1, pick).view(case["tokens"], case["choices"])


def _sorted(expert_of, experts):
    """(row of every choice, choice of every row, offsets): rows by expert, within an expert in the choices' order; -1
    where a choice has no row and where a row behind the last expert's has no choice."""
    flat = expert_of.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    offsets = torch.searchsorted(key[order], torch.arange(experts + 1, device=key.device))
    row_of = torch.where(key < experts, place, -1).view(expert_of.shape)
    choice_of = torch.where(torch.arange(order.numel(), device=order.device) < offsets[-1], order, -1)
    return row_of.to(torch.int32), choice_of.to(torch.int32), offsets.to(torch.int32)


def _tensor_sizes(case):
    """Sizes of a transformer's parameters: embeddings of `words` words, then `layers` layers of hidden width h with
    four projections and a feed-forward part four times as wide, each with its bias, and two norms."""
    h, sizes = case["hidden"], []
    if case["words"]:
        sizes += [case["words"] * h, 512 * h, 2 * h, h, h]
    for _ in range(case["layers"]):
        sizes += [h * h, h] * 4 + [h, h, 4 * h * h, 4 * h, 4 * h * h, h, h, h]
    return sizes


def _views(flat, sizes):
    """Tensors of these sizes in one buffer, each from a multiple of 16 elements on."""
    at, out = 0, []
    for n in sizes:
        out.append(flat[at:at + n])
        at += -(-n // 16) * 16
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("clip", "reduce_clip"):
        sizes, ranks = _tensor_sizes(case), case["ranks"]
        total = sum(-(-n // 16) * 16 for n in sizes)
        s["sizes"] = sizes
        s["grads"] = torch.empty(ranks, total, dtype=DTYPES[case["dtype"]], device="cuda")
        for r in range(ranks):
            s["grads"][r] = torch.randn(total, generator=g, device="cuda").mul_(GRAD)
        # (what lies between the tensors is none of them)
        used = torch.zeros(total, dtype=torch.bool, device="cuda")
        for v in _views(used, sizes):
            v.fill_(True)
        s["grads"].masked_fill_(~used, 0.0)
        s["out"] = torch.zeros(ranks if op == "clip" else 1, total, dtype=DTYPES[case["out"]], device="cuda")
        s["norm"] = torch.empty(1, device="cuda")
        # what the norm is about, times `share`: half of it is clipped to, twice of it never reached
        values = sum(sizes) * (ranks if op == "clip" else 1.0 / ranks)
        s["max_norm"] = case["share"] * GRAD * values ** 0.5
        if own:  # the tables of the tensors' addresses, built once for a training run
            from collective_fusedallreduce_gb300 import coco

            for name in ("grads", "out"):
                per_rank = [_views(row, sizes) for row in s[name]]
                s[name + "_table"] = torch.empty(coco.coco_scattered_table_bytes(sizes, len(per_rank)),
                                                 dtype=torch.uint8, device="cuda")
                s[name + "_plan"] = coco.coco_scattered_table_build(per_rank, s[name + "_table"])
        return s
    dt, cols = DTYPES[case["dtype"]], case["cols"]
    if op in ("norm", "norm_grad"):
        ranks, rows = case["ranks"], case["rows"]
        s["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(dt)
        s["bias"] = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(dt)
    else:
        tokens, choices = case["tokens"], case["choices"]
    if op == "norm":
        s["partials"] = _activations(g, (ranks, rows, cols), dt, ranks ** -0.5)
        s["residual"] = _activations(g, (rows, cols), dt)
        out = DTYPES["fp8"] if case["out"] == "fp8" else dt
        n = case["copies"]
        s["hidden"] = [torch.empty(rows, cols, dtype=dt, device="cuda") for _ in range(n)]
        s["normed"] = [torch.empty(rows, cols, dtype=out, device="cuda") for _ in range(n)]
        s["scales"] = [torch.empty(rows, _blocks(cols), device="cuda") for _ in range(n)] \
            if case["out"] == "fp8" else None
        s["mean"], s["rstd"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    elif op == "norm_grad":
        s["dnormed"] = (torch.randn(ranks, rows, cols, generator=g, device="cuda") * ranks ** -0.5).to(dt)
        s["dhidden"] = torch.randn(rows, cols, generator=g, device="cuda").to(dt)
        s["hidden"] = _activations(g, (rows, cols), dt)
        h = s["hidden"].float()
        s["mean"] = h.mean(-1)
        s["rstd"] = (h.var(-1, correction=0) + EPS).rsqrt()
        s["dx"] = torch.empty(rows, cols, dtype=dt, device="cuda")
        s["dweight"], s["dbias"] = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    elif op == "dispatch":
        experts, n = case["experts"], tokens * choices
        x = _activations(g, (tokens, cols), torch.float32)
        fp8 = case["dtype"] == "fp8"
        s["x"], s["scales"] = _held_in_8_bits(x) if fp8 else (x.to(dt), None)
        s["expert_of"] = _routing(g, case, experts, case["skew"])
        s["row_of"] = torch.empty(tokens, choices, dtype=torch.int32, device="cuda")
        s["choice_of"] = torch.empty(n, dtype=torch.int32, device="cuda")
        s["offsets"] = torch.empty(1, experts + 1, dtype=torch.int32, device="cuda")
        s["rows"] = torch.zeros(n, cols, device="cuda").to(dt)
        s["row_scales"] = torch.zeros(n, _blocks(cols), device="cuda") if fp8 else None
    else:
        ranks, experts = case["ranks"], 32
        s["row_of"] = _sorted(_routing(g, case, experts, 1.0), experts)[0]
        s["rows"] = _activations(g, (ranks, tokens * choices, cols), dt, ranks ** -0.5)
        weights = torch.rand(tokens, choices, generator=g, device="cuda").add_(0.1)
        s["gates"] = weights / weights.sum(-1, keepdim=True) if case.get("weights", True) else None
        if op == "combine":
            s["residual"] = _activations(g, (tokens, cols), dt) if case["summed"] else None
            s["out"] = torch.empty(1 if case["summed"] else ranks, tokens, cols, dtype=dt, device="cuda")
        else:
            s["dout"] = torch.randn(tokens, cols, generator=g, device="cuda").to(dt)
            s["drows"] = torch.zeros(tokens * choices, cols, dtype=dt, device="cuda")
            s["dgates"] = torch.empty(tokens, choices, device="cuda")
    return s


def run(s):
    return _framework(s) if own else _plain(s)


# ------------------------------------------------------------------------------ the framework's calls


def _framework(s):
    from collective_fusedallreduce_gb300 import coco

    case = s["case"]
    op = case["op"]
    if op == "dispatch":
        coco.coco_expert_sort(s["expert_of"], case["experts"], s["row_of"], s["choice_of"], s["offsets"])
        fp8 = case["dtype"] == "fp8"
        coco.coco_expert_dispatch(coco.replicated([s["x"]]), [s["scales"]] if fp8 else None, s["row_of"],
                                  coco.replicated([s["rows"]]), [s["row_scales"]] if fp8 else None)
        return {"row_of": s["row_of"], "choice_of": s["choice_of"], "offsets": s["offsets"], "rows": s["rows"],
                "row_scales": s["row_scales"]}
    if op == "combine":
        n = case["ranks"]
        if case["summed"]:
            coco.coco_expert_combine(coco.local(list(s["rows"])), s["row_of"], s["gates"],
                                     coco.replicated([s["residual"]] * n), coco.replicated([s["out"][0]] * n))
        else:
            coco.coco_expert_combine(coco.local(list(s["rows"])), s["row_of"], s["gates"], None,
                                     coco.local(list(s["out"])))
        return s["out"]
    if op == "combine_grad":
        n = case["ranks"]
        coco.coco_expert_combine_backward(coco.replicated([s["dout"]] * n), coco.local(list(s["rows"])), s["row_of"],
                                          s["gates"], coco.replicated([s["drows"]] * n), s["dgates"])
        return {"drows": s["drows"], "dgates": s["dgates"]}
    if op == "norm":
        n, copies = case["ranks"], case["copies"]
        spread = (lambda v: v) if copies == n else (lambda v: v * n)  # a copy for every rank, or one for all
        coco.coco_allreduce_layernorm(
            coco.local(list(s["partials"])), coco.replicated([s["residual"]] * n), s["weight"], s["bias"], EPS,
            coco.replicated(spread(s["hidden"])), coco.replicated(spread(s["normed"])),
            spread(s["scales"]) if s["scales"] else None, s["mean"], s["rstd"])
        return {"hidden": s["hidden"], "normed": s["normed"], "scales": s["scales"], "mean": s["mean"],
                "rstd": s["rstd"]}
    if op == "norm_grad":
        n, rows, cols = case["ranks"], case["rows"], case["cols"]
        space = torch.empty(coco.coco_allreduce_layernorm_backward_bytes(rows, cols), dtype=torch.uint8,
                            device="cuda")
        coco.coco_allreduce_layernorm_backward(
            coco.local(list(s["dnormed"])), coco.replicated([s["dhidden"]] * n), coco.replicated([s["hidden"]] * n),
            s["weight"], s["mean"], s["rstd"], coco.replicated([s["dx"]] * n), s["dweight"], s["dbias"], space)
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    space = torch.empty(coco.coco_scattered_clip_bytes(), dtype=torch.uint8, device="cuda")
    if op == "clip":
        coco.coco_scattered_clip(s["grads_plan"], coco.LOCAL, s["max_norm"], s["out_plan"], s["norm"], space)
    else:
        coco.coco_scattered_allreduce_clip(s["grads_plan"], 1.0 / case["ranks"], s["max_norm"], s["out_plan"],
                                           s["norm"], space)
    return {"out": s["out"], "norm": s["norm"]}


# ------------------------------------------------------------------------------------- the plain form


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "dispatch":
        row_of, choice_of, offsets = _sorted(s["expert_of"], case["experts"])
        live = (choice_of >= 0)[:, None]
        token = choice_of.clamp_min(0).long() // case["choices"]
        if case["dtype"] == "fp8":
            held = torch.where(live, s["x"].view(torch.uint8)[token], 0).view(torch.float8_e4m3fn)
            return {"row_of": row_of, "choice_of": choice_of, "offsets": offsets[None], "rows": held,
                    "row_scales": torch.where(live, s["scales"][token], 0.0)}
        return {"row_of": row_of, "choice_of": choice_of, "offsets": offsets[None],
                "rows": torch.where(live, s["x"][token], 0.0), "row_scales": None}
    if op == "combine":
        at = s["row_of"].clamp_min(0).long()
        weight = (s["row_of"] >= 0).float() if s["gates"] is None else torch.where(s["row_of"] >= 0, s["gates"], 0.0)
        if case["summed"]:
            rows = s["rows"].sum(0, dtype=torch.float32)
            out = (rows[at] * weight[..., None]).sum(1) + s["residual"].float()
            return out.to(s["out"].dtype)[None]
        return (s["rows"][:, at].float() * weight[..., None]).sum(2).to(s["out"].dtype)
    if op == "combine_grad":
        live, at, dout = s["row_of"] >= 0, s["row_of"].clamp_min(0).long(), s["dout"].float()
        rows = s["rows"].sum(0, dtype=torch.float32)
        dgates = torch.where(live, (rows[at] * dout[:, None]).sum(-1), 0.0)
        drows = torch.zeros(s["drows"].shape, dtype=torch.float32, device="cuda")
        parts = s["gates"][..., None] * dout[:, None]
        drows[s["row_of"][live].long()] = parts[live]
        return {"drows": drows.to(s["drows"].dtype), "dgates": dgates}
    if op == "norm":
        h = s["partials"].sum(0, dtype=torch.float32) + s["residual"].float()
        mean = h.mean(-1)
        centred = h - mean[:, None]
        rstd = (centred.square().mean(-1) + EPS).rsqrt()
        y = centred * rstd[:, None] * s["weight"].float() + s["bias"].float()
        dt = s["residual"].dtype
        copies = case["copies"]
        q, scales = _held_in_8_bits(y) if case["out"] == "fp8" else (y.to(dt), None)
        return {"hidden": [h.to(dt) for _ in range(copies)], "normed": [q.clone() for _ in range(copies)],
                "scales": [scales.clone() for _ in range(copies)] if scales is not None else None, "mean": mean,
                "rstd": rstd}
    if op == "norm_grad":
        dy, r = s["dnormed"].sum(0, dtype=torch.float32), s["rstd"][:, None]
        xhat = (s["hidden"].float() - s["mean"][:, None]) * r
        g = dy * s["weight"].float()
        dx = r * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True)) + s["dhidden"].float()
        return {"dx": dx.to(s["hidden"].dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}
    # (the buffers' gaps are zeros, so the tensors can be taken together)
    if op == "clip":
        x = s["grads"].float()
    else:
        x = (s["grads"].sum(0, dtype=torch.float32) * (1.0 / case["ranks"])).to(s["out"].dtype).float()[None]
    norm = x.square().sum(dtype=torch.float64).sqrt()
    factor = torch.where(norm <= s["max_norm"], 1.0, s["max_norm"] / norm).float()
    return {"out": (x * factor).to(s["out"].dtype), "norm": norm.float()[None]}


# --------------------------------------------------------------------------- the definitions in 64 bits


def _e4m3_of(y):
    """(values on the e4m3 grid, scales) of rows in 64 bits, block by block of columns."""
    rows, cols = y.shape
    values, scales = torch.empty_like(y), y.new_empty(rows, _blocks(cols))
    for b in range(_blocks(cols)):
        part = y[:, b * BLOCK:(b + 1) * BLOCK]
        sc = part.abs().amax(-1).clamp_min(2.0 ** -100) / E4M3_MAX
        scales[:, b] = sc
        v = part / sc[:, None]
        # e4m3: three fraction bits above 2^-6, steps of 2^-9 below
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))).clamp_min(-6) - 3)
        values[:, b * BLOCK:(b + 1) * BLOCK] = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    return values, scales


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        # a row per choice, expert by expert: whole numbers have no other value than their own
        flat, x = s["expert_of"].reshape(-1), s["x"].float()
        of_choice = torch.arange(case["tokens"], device="cuda").repeat_interleave(case["choices"])
        rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device="cuda")
        scales = None if s["scales"] is None else torch.zeros(s["row_scales"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for e in range(case["experts"]):
            picked = of_choice[flat == e]
            n = picked.numel()
            rows[at:at + n] = x[picked].double()
            if scales is not None:
                scales[at:at + n] = s["scales"][picked].double()
            at += n
        return {"row_of": None, "choice_of": None, "offsets": None, "rows": rows, "row_scales": scales}
    if op in ("combine", "combine_grad"):
        tokens, choices, cols = case["tokens"], case["choices"], case["cols"]
        one = torch.ones(tokens, choices, dtype=torch.float64, device="cuda")
        gates = one if s["gates"] is None else s["gates"].double()
        token = torch.arange(tokens, device="cuda")
        if op == "combine":
            out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
            for r in range(case["ranks"]):
                to = out[0 if case["summed"] else r]
                for k in range(choices):
                    has = s["row_of"][:, k] >= 0
                    part = s["rows"][r][s["row_of"][has, k].long()].double()
                    to.index_add_(0, token[has], part * gates[has, k][:, None])
            return out + s["residual"].double() if case["summed"] else out
        drows = torch.zeros(tokens * choices, cols, dtype=torch.float64, device="cuda")
        dgates = torch.zeros(tokens, choices, dtype=torch.float64, device="cuda")
        for k in range(choices):
            has = s["row_of"][:, k] >= 0
            at, d = s["row_of"][has, k].long(), s["dout"][has].double()
            drows[at] = torch.einsum("t,tc->tc", gates[has, k], d)
            for r in range(case["ranks"]):
                dgates[has, k] += torch.einsum("tc,tc->t", d, s["rows"][r][at].double())
        return {"drows": drows, "dgates": dgates}
    if op == "norm":
        h = s["residual"].double()
        for p in s["partials"]:
            h = h + p.double()
        mean = torch.einsum("rc->r", h) / case["cols"]
        h0 = h - mean[:, None]
        rstd = 1.0 / torch.sqrt(torch.einsum("rc,rc->r", h0, h0) / case["cols"] + EPS)
        y = torch.einsum("rc,r,c->rc", h0, rstd, s["weight"].double()) + s["bias"].double()
        copies = case["copies"]
        q, scales = _e4m3_of(y) if case["out"] == "fp8" else (y, None)
        return {"hidden": [h] * copies, "normed": [q] * copies,
                "scales": [scales] * copies if scales is not None else None, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        dy = sum(p.double() for p in s["dnormed"])
        h0, r, w = s["hidden"].double() - s["mean"].double()[:, None], s["rstd"].double(), s["weight"].double()
        # (h - mean) r w's derivative: w r dy, less its row's mean, less (h - mean) r^3 / C times their product
        along = torch.einsum("rc,c,rc->r", dy, w, h0)
        dx = (dy * w - (torch.einsum("rc,c->r", dy, w) / case["cols"])[:, None]) * r[:, None]
        dx = dx - h0 * (r ** 3 * along / case["cols"])[:, None] + s["dhidden"].double()
        return {"dx": dx, "dweight": torch.einsum("rc,rc,r->c", dy, h0, r), "dbias": dy.sum(0)}
    n, total = len(s["out"]), s["out"].shape[1]
    out = torch.zeros(n, total, dtype=torch.float64, device="cuda")
    for r, row in enumerate(s["grads"]):
        for to, x in zip(_views(out[r if op == "clip" else 0], s["sizes"]), _views(row, s["sizes"])):
            to += x.double() / (1 if op == "clip" else case["ranks"])
    norm = torch.linalg.vector_norm(out)
    if norm > s["max_norm"]:
        out *= s["max_norm"] / norm
    return {"out": out, "norm": norm[None]}


# -------------------------------------------------------------------------------------- the work of a pass


def work(case):
    """Each input read once and each output written once; two operations for a product's multiply and add."""
    op = case["op"]
    es = SIZES[case["dtype"]]
    if op in ("clip", "reduce_clip"):
        n, ranks = sum(_tensor_sizes(case)), case["ranks"]
        written = n * (ranks if op == "clip" else 1)
        return {"bytes": n * ranks * es + written * SIZES[case["out"]], "flops": n * ranks + 3 * written}
    cols = case["cols"]
    if op == "norm":
        v = case["rows"] * cols
        out = v + 4 * case["rows"] * _blocks(cols) if case["out"] == "fp8" else v * es
        return {"bytes": v * es * (case["ranks"] + 1) + 2 * cols * es + case["copies"] * (v * es + out)
                + 8 * case["rows"], "flops": v * (case["ranks"] + 8)}
    if op == "norm_grad":
        v = case["rows"] * cols
        return {"bytes": v * es * (case["ranks"] + 3) + cols * (es + 8) + 8 * case["rows"],
                "flops": v * (case["ranks"] + 14)}
    n = case["tokens"] * case["choices"]
    kept = n * (1.0 - case["dropped"])
    if op == "dispatch":
        row = cols * es + (4 * _blocks(cols) if case["dtype"] == "fp8" else 0)
        return {"bytes": (case["tokens"] + kept) * row + n * (8 + 4 + 4) + 4 * (case["experts"] + 1), "flops": n}
    ranks, v = case["ranks"], case["tokens"] * cols
    if op == "combine":
        around = 2 * v if case["summed"] else ranks * v
        return {"bytes": es * (ranks * kept * cols + around) + n * (8 if case["weights"] else 4),
                "flops": kept * cols * (ranks + 1)}
    return {"bytes": es * ((ranks + 1) * kept * cols + v) + n * 12, "flops": kept * cols * (ranks + 3)}
