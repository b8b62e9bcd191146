"""Cases that measure what follows a router: tokens sorted by expert, gathered to their experts and brought back
with their weights (and the gradients), blocks of 128 quantised to 8-bit floats, and the experts' products of such
operands."""
import torch

own = False

SIZES = {"bf16": 2, "fp32": 4, "e4m3": 1, "e5m2": 1}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
BLOCK = 128
LEAST = 2.0 ** -100  # the smallest magnitude that a block's scale is made for


def _routed(name, op, tokens, k, experts, align=1, dropped=0.0, **more):
    return {"name": name, "op": op, "tokens": tokens, "k": k, "experts": experts, "align": align, "dropped": dropped,
            **more}


def listed():
    return [
        # one decode step of a small batch: latency
        _routed("sort decode 4x8 of 256", "sort", 4, 8, 256),
        # a training micro-batch, segments of whole blocks of 128
        _routed("sort train 65536x8 of 256", "sort", 65536, 8, 256, 128),
        # the hidden rows of a training micro-batch to their experts
        _routed("gather train 8192x8 x 4096", "gather", 8192, 8, 64, 128, n=4096, dtype="bf16"),
        # odd sizes, some slots dropped by a capacity limit, 32 bits
        _routed("gather odd 517x6 x 1001", "gather", 517, 6, 61, 1, 0.05, n=1001, dtype="fp32"),
        # the experts' results back to their tokens
        _routed("combine train 8192x8 x 4096", "combine", 8192, 8, 64, 128, n=4096, dtype="bf16", grad=False),
        # a decode step: latency
        _routed("combine decode 4x8 x 2048", "combine", 4, 8, 256, n=2048, dtype="fp32", grad=False),
        # the gradients of the experts' results and of the weights
        _routed("combine grad 8192x8 x 4096", "combine", 8192, 8, 64, 128, n=4096, dtype="bf16", grad=True),
        # the hidden rows to their experts as 8-bit operands of the first product
        _routed("quantize rows 8192x8 x 4096", "quantize", 8192, 8, 64, 128, n=4096, dtype="bf16", to="e4m3",
                layout="row"),
        # the same rows transposed, in blocks of 128 tokens, for the weights' gradient: odd sizes, 32 bits
        _routed("quantize columns 4099x6 x 2001", "quantize", 4099, 6, 61, 128, 0.05, n=2001, dtype="fp32", to="e5m2",
                layout="column"),
        # the experts' product of a decode step: the weights of the experts that were hit are read once
        _routed("product decode 4x8 of 64", "product", 4, 8, 64, kind="rows", n=2048, inner=4096, a="e4m3", b="tile",
                out="bf16"),
        # the experts' product of a training micro-batch, ragged loads
        _routed("product train 8192x8 of 64", "product", 8192, 8, 64, 128, kind="rows", n=4096, inner=4096, a="e4m3",
                b="tile", out="bf16"),
        # the weights' gradients: a product along each expert's tokens, operands in blocks of 128 tokens
        _routed("product inner 8192x4 of 16", "product", 8192, 4, 16, 128, kind="inner", n=2048, m=4096, a="e5m2",
                b="row", out="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["sort", "gather", "combine", "combine", "quantize", "quantize", "product", "product", "product"])
    experts = _log(rng, 2, 256)
    k = rng.randint(1, min(8, experts))
    align, dropped = rng.choice([1, 1, 16, 128]), rng.choice([0.0, 0.0, 0.05])
    tokens = _log(rng, 1, 65536 if op == "sort" else 8192)
    if op == "sort":
        c = _routed("", op, tokens, k, experts, align, dropped)
    elif op in ("gather", "combine"):
        c = _routed("", op, tokens, k, experts, align, dropped, n=_log(rng, 32, 4096), dtype=rng.choice(["bf16", "fp32"]))
        if op == "combine":
            c["grad"] = rng.random() < 0.5
    elif op == "quantize":
        layout = rng.choice(["row", "row", "column", "tile"])
        n = _log(rng, 32, 4096)
        c = _routed("", op, tokens, k, experts, 128 if layout == "column" else align, dropped, n=n,
                    dtype=rng.choice(["bf16", "fp32"]), to=rng.choice(["e4m3", "e5m2"]), layout=layout)
    else:
        kind = rng.choice(["none", "rows", "rows", "inner"])
        tokens, experts = _log(rng, 1, 4096), min(experts, 64)
        c = _routed("", op, tokens, k, experts, 128 if kind == "inner" else align, dropped, kind=kind,
                    n=_log(rng, 64, 4096), inner=16 * _log(rng, 4, 256), a=rng.choice(["e4m3", "e5m2"]),
                    b="row" if kind == "inner" else rng.choice(["tile", "tile", "row"]), out=rng.choice(["bf16", "fp32"]))
        if kind == "inner":
            c["m"], c["n"] = _log(rng, 64, 2048), min(c["n"], 2048)
            del c["inner"]
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------- inputs
def _capacity(slots, experts, align):
    """Positions that hold any choice of experts: each segment with a slot can end in align - 1 positions of padding."""
    return (slots + min(slots, experts) * (align - 1)) // align * align


def _choices(g, case):
    """The experts of every token, as a router with an uneven load gives them; dropped slots hold -1."""
    T, E, k = case["tokens"], case["experts"], case["k"]
    x = torch.randn(T, E, generator=g, device="cuda") + 0.3 * torch.randn(E, generator=g, device="cuda")
    idx = x.topk(k, dim=1)[1].to(torch.int32)
    if case["dropped"]:
        idx[torch.rand(T, k, generator=g, device="cuda") < case["dropped"]] = -1
    return idx.contiguous()


def _sorted(idx, E, align):
    """place [tokens, k], order [capacity], offsets [experts + 1], all int32."""
    T, k = idx.shape
    key = torch.where((idx < 0) | (idx >= E), E, idx).reshape(-1).long()
    counts = torch.zeros(E + 1, dtype=torch.long, device=idx.device).scatter_add_(0, key, torch.ones_like(key))
    ends = ((counts[:E] + align - 1) // align * align).cumsum(0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    by_expert, slot = key.sort(stable=True)
    first = counts.cumsum(0) - counts
    at = torch.arange(T * k, device=idx.device)
    pos = torch.where(by_expert < E, offsets[by_expert.clamp(max=E)] + at - first[by_expert], -1)
    place = torch.empty_like(key).scatter_(0, slot, pos)
    cap = _capacity(T * k, E, align)
    order = torch.full((cap + 1,), -1, dtype=torch.long, device=idx.device).scatter_(
        0, torch.where(pos < 0, cap, pos), slot)[:cap]
    return place.view(T, k).to(torch.int32), order.to(torch.int32), offsets.to(torch.int32)


def _quantized(x, to, rows, pad=0):
    """x [.., r, n] in blocks of rows x 128: the 8-bit values and the scales."""
    r, n = x.shape[-2:]
    up = torch.nn.functional.pad(x.float(), (0, -n % BLOCK, 0, -r % rows))
    tiles = up.view(*x.shape[:-2], up.shape[-2] // rows, rows, up.shape[-1] // BLOCK, BLOCK)
    scales = tiles.abs().amax(dim=(-3, -1)).clamp(min=LEAST) / LARGEST[to]
    q = (tiles / scales[..., :, None, :, None]).reshape(up.shape)[..., :r, :n]
    return torch.nn.functional.pad(q, (0, pad)).to(TYPES[to]), scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    op, T, E, k = case["op"], case["tokens"], case["experts"], case["k"]
    s = {"case": case, "idx": _choices(g, case)}
    if op == "sort":
        return s
    s["place"], s["order"], s["offsets"] = _sorted(s["idx"], E, case["align"])
    cap = s["order"].numel()
    if op == "gather":
        s["x"] = randn(T, case["n"]).to(TYPES[case["dtype"]])
        s["out"] = torch.zeros(cap, case["n"], dtype=s["x"].dtype, device="cuda")
    elif op == "combine":
        dt = TYPES[case["dtype"]]
        s["y"] = randn(cap, case["n"]).to(dt)
        s["w"] = torch.rand(T, k, generator=g, device="cuda")
        s["w"] /= s["w"].sum(dim=1, keepdim=True)
        if case["grad"]:
            s["g"] = randn(T, case["n"]).to(dt)
            s["out"] = torch.zeros(cap, case["n"], dtype=dt, device="cuda")
    elif op == "quantize":
        # channels of uneven size, as hidden rows have
        s["x"] = (randn(T, case["n"]) * torch.exp(randn(case["n"]))).to(TYPES[case["dtype"]])
        wide = -(-case["n"] // 16) * 16
        if case["layout"] == "row":
            s["out"] = torch.zeros(cap, wide, device="cuda").to(TYPES[case["to"]])
            s["scales"] = torch.zeros(cap, -(-case["n"] // BLOCK), device="cuda")
        elif case["layout"] == "column":
            s["out"] = torch.zeros(case["n"], -(-cap // 16) * 16, device="cuda").to(TYPES[case["to"]])
            s["scales"] = torch.zeros(case["n"], -(-cap // BLOCK), device="cuda")
    else:
        n, a, of_b = case["n"], case["a"], 128 if case["b"] == "tile" else 1
        # the longest segment, which the plain form's batched product is padded to
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        if case["kind"] == "inner":
            x = randn(cap, case["m"] + n)
            x[s["order"] < 0] = 0
            x = x.t().contiguous()
            s["a"], s["sa"] = _quantized(x[:case["m"]], a, 1, -cap % 16)
            s["b"], s["sb"] = _quantized(x[case["m"]:], "e4m3", 1, -cap % 16)
        else:
            grouped = case["kind"] == "rows"
            rows = cap if grouped else T
            x = randn(rows, case["inner"])
            if grouped:
                x[s["order"] < 0] = 0
                s["out"] = torch.zeros(rows, n, dtype=TYPES[case["out"]], device="cuda")
            s["a"], s["sa"] = _quantized(x, a, 1)
            w = randn(E, n, case["inner"]) if grouped else randn(n, case["inner"])
            s["b"], s["sb"] = _quantized(w * case["inner"] ** -0.5, "e4m3", of_b)
    return s


# ----------------------------------------------------------------------------------- plain forms
def _rows_of(order, k):
    return (order.long() // k).clamp(min=0)


def _plain_sort(s, c):
    return _sorted(s["idx"], c["experts"], c["align"])


def _plain_gather(s, c):
    return torch.where(s["order"][:, None] < 0, 0, s["x"][_rows_of(s["order"], c["k"])])


def _plain_combine(s, c):
    place, y, w = s["place"].long(), s["y"], s["w"]
    hole = place < 0
    rows = torch.where(hole[:, :, None], 0, y[place.clamp(min=0)].float())
    if not c["grad"]:
        return (torch.where(hole, 0, w)[:, :, None] * rows).sum(dim=1).to(y.dtype)
    of = s["order"]
    at = of.long().clamp(min=0)
    grad_w = (s["g"].float()[:, None, :] * rows).sum(dim=2)
    grad_y = torch.where(of < 0, 0, w.reshape(-1)[at])[:, None] * s["g"][at // c["k"]].float()
    return grad_y.to(y.dtype), grad_w


def _plain_quantize(s, c):
    x, wide = s["x"], -c["n"] % 16
    if c["layout"] == "tile":
        return _quantized(x, c["to"], BLOCK, wide)
    rows = torch.where(s["order"][:, None] < 0, 0, x[_rows_of(s["order"], c["k"])])
    if c["layout"] == "column":
        rows, wide = rows.t(), -rows.shape[0] % 16
    q, scales = _quantized(rows, c["to"], 1, wide)
    # rows (columns) behind the last segment are nobody's
    live = torch.arange(s["order"].numel(), device=x.device) < s["offsets"][-1]
    if c["layout"] == "column":
        live = live[::BLOCK]
        return q, torch.where(live[None], scales, 0)
    return q, torch.where(live[:, None], scales, 0)


def _values(q, scales, rows):
    """The numbers that 8-bit values and their blocks' scales stand for."""
    each = scales.repeat_interleave(rows, dim=-2)[..., :q.shape[-2], :].repeat_interleave(BLOCK, dim=-1)
    return q.float() * each[..., :q.shape[-1]]


def _plain_product(s, c):
    of_b, out = 128 if c["b"] == "tile" else 1, TYPES[c["out"]]
    if c["kind"] == "none":
        return (_values(s["a"], s["sa"], 1) @ _values(s["b"], s["sb"], of_b).t()).to(out)
    offsets, cap = s["offsets"].long(), s["order"].numel()
    at = offsets[:-1, None] + torch.arange(s["most"], device=offsets.device)[None]  # [experts, most]
    live = at < offsets[1:, None]
    at = torch.where(live, at, 0)
    if c["kind"] == "inner":
        a = torch.where(live[:, None], _values(s["a"], s["sa"], 1)[:, at].transpose(0, 1), 0)
        b = torch.where(live[:, :, None], _values(s["b"], s["sb"], 1).t()[at], 0)
        return torch.bmm(a, b).to(out)
    a = _values(s["a"], s["sa"], 1)
    if cap <= 64:  # a few rows: each with its own expert's weights
        expert = (torch.arange(cap, device=a.device)[:, None] >= offsets[None, 1:]).sum(dim=1).clamp(max=c["experts"] - 1)
        full = torch.bmm(_values(s["b"][expert], s["sb"][expert], of_b), a[:, :, None])[:, :, 0]
    else:
        b = _values(s["b"], s["sb"], of_b)
        each = torch.bmm(a[at], b.transpose(1, 2).contiguous())
        full = a.new_zeros(cap + 1, c["n"])
        full[torch.where(live, at, cap)] = each
        full = full[:cap]
    return torch.where(torch.arange(cap, device=a.device)[:, None] < offsets[-1], full, 0).to(out)


def _own(s, c):
    import top_selection_amd as ts
    op = c["op"]
    if op == "sort":
        p = ts.ds_expert_sort(s["idx"], c["experts"], align=c["align"])
        return p.place, p.order, p.offsets
    plan = ts.ExpertPlan(s["place"], s["order"], s["offsets"], c["align"])
    if op == "gather":
        return ts.ds_expert_gather(s["x"], plan, out=s["out"])
    if op == "combine":
        if not c["grad"]:
            return ts.ds_expert_combine(s["y"], plan, s["w"])
        return ts.ds_expert_combine_grad(s["g"], s["y"], plan, s["w"], out_y=s["out"])
    if op == "quantize":
        to = TYPES[c["to"]]
        if c["layout"] == "tile":
            return ts.ds_block_quantize(s["x"], ts.BLOCK_TILE, dtype=to)
        layout = ts.BLOCK_ROW if c["layout"] == "row" else ts.BLOCK_COLUMN
        return ts.ds_block_quantize(s["x"], layout, dtype=to, plan=plan, out=s["out"], out_scales=s["scales"])
    if c["kind"] == "none":
        return ts.ds_block_product(s["a"], s["sa"], s["b"], s["sb"], out_dtype=TYPES[c["out"]])
    if c["kind"] == "inner":
        return ts.ds_block_product(s["a"], s["sa"], s["b"], s["sb"], offsets=s["offsets"], inner=True,
                                   out_dtype=TYPES[c["out"]])
    return ts.ds_block_product(s["a"], s["sa"], s["b"], s["sb"], offsets=s["offsets"], out=s["out"])


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return {"sort": _plain_sort, "gather": _plain_gather, "combine": _plain_combine, "quantize": _plain_quantize,
            "product": _plain_product}[c["op"]](state, c)


def work(case):
    op, T, E, k = case["op"], case["tokens"], case["experts"], case["k"]
    slots = T * k
    # an even share of the padding: half of the alignment for each expert that has a slot
    hit = E * (1 - (1 - k / E) ** T)
    total = int(slots * (1 - case["dropped"]) + hit * (case["align"] - 1) / 2)
    if op == "sort":
        return {"bytes": 4 * (2 * slots + _capacity(slots, E, case["align"]) + E + 1), "flops": slots}
    n = case["n"]
    if op == "gather":
        return {"bytes": (T + total) * n * SIZES[case["dtype"]] + 8 * slots, "flops": 0}
    live = int(slots * (1 - case["dropped"]))
    if op == "combine":
        b = SIZES[case["dtype"]]
        if case["grad"]:
            return {"bytes": (T + live + total) * n * b + 16 * slots, "flops": 3 * live * n}
        return {"bytes": (T + live) * n * b + 8 * slots, "flops": 2 * live * n}
    if op == "quantize":
        if case["layout"] == "tile":
            return {"bytes": T * n * (SIZES[case["dtype"]] + 1) + T * n // 4096, "flops": 4 * T * n}
        return {"bytes": T * n * SIZES[case["dtype"]] + total * n + total * n // 32 + 8 * slots, "flops": 4 * total * n}
    o = SIZES[case["out"]]
    if case["kind"] == "none":
        i = case["inner"]
        return {"bytes": (T + n) * i + T * i // 32 + T * n * o, "flops": 2 * T * n * i}
    if case["kind"] == "rows":
        i = case["inner"]
        return {"bytes": int(hit * n * i) + total * (i + i // 32 + n * o), "flops": 2 * live * n * i}
    return {"bytes": (case["m"] + n) * total * 33 // 32 + E * case["m"] * n * o, "flops": 2 * live * n * case["m"]}


# ------------------------------------------------------------------- the definitions in 64 bits
def _round8(v, to):
    """To the nearest 8-bit float, ties to even, for magnitudes up to the largest."""
    bits, least = (3, -6) if to == "e4m3" else (2, -14)
    exponent = torch.frexp(v.abs())[1].long() - 1
    step = torch.exp2((exponent.clamp(min=least) - bits).double())
    return torch.round(v / step) * step


def _exact_quantize(x, to, case):
    """x [rows, n] in 64 bits, blocks of 128 along its rows."""
    r, n = x.shape
    q = x.new_zeros(r, -(-n // 16) * 16)
    scales = x.new_zeros(r, -(-n // BLOCK))
    for j in range(scales.shape[1]):
        part = x[:, j * BLOCK:(j + 1) * BLOCK]
        scales[:, j] = part.abs().amax(dim=1).clamp(min=LEAST) / LARGEST[to]
        # the definition divides by the scale that is stored
        q[:, j * BLOCK:j * BLOCK + part.shape[1]] = _round8(part / scales[:, j:j + 1].float().double(), to)
    return q, scales


def exact(case, seed):
    """Expert by expert and slot by slot, from the definitions."""
    import numpy as np
    op, E, k, align = case["op"], case["experts"], case["k"], case["align"]
    s = prepare(case, seed)
    idx = s["idx"].cpu().numpy().reshape(-1)
    order, offsets = np.full(_capacity(idx.size, E, align), -1, np.int32), np.zeros(E + 1, np.int32)
    place = np.full(idx.size, -1, np.int32)
    for e in range(E):
        mine = np.flatnonzero(idx == e)
        order[offsets[e]:offsets[e] + mine.size] = mine
        place[mine] = offsets[e] + np.arange(mine.size)
        offsets[e + 1] = offsets[e] + -(-mine.size // align) * align
    if op == "sort":
        return place.reshape(-1, k), order, offsets
    total, cap = int(offsets[E]), order.size
    slot = torch.from_numpy(np.flatnonzero(order >= 0)).cuda()  # positions that hold a slot
    token = torch.from_numpy(order[order >= 0].astype(np.int64) // k).cuda()
    if op == "gather":
        out = torch.zeros(cap, case["n"], dtype=torch.float64, device="cuda")
        out[slot] = s["x"][token].double()
        return out
    if op == "combine":
        w = s["w"].double().reshape(-1)[torch.from_numpy(order[order >= 0].astype(np.int64)).cuda()]
        if not case["grad"]:
            out = torch.zeros(case["tokens"], case["n"], dtype=torch.float64, device="cuda")
            for j in range(k):
                at = torch.from_numpy(place.reshape(-1, k)[:, j].astype(np.int64)).cuda()
                has = at >= 0
                out[has] += s["w"][has, j, None].double() * s["y"][at[has]].double()
            return out
        grad_y = torch.zeros(cap, case["n"], dtype=torch.float64, device="cuda")
        grad_y[slot] = w[:, None] * s["g"][token].double()
        grad_w = torch.zeros(case["tokens"], k, dtype=torch.float64, device="cuda")
        for j in range(k):
            at = torch.from_numpy(place.reshape(-1, k)[:, j].astype(np.int64)).cuda()
            has = at >= 0
            grad_w[has, j] = (s["g"][has].double() * s["y"][at[has]].double()).sum(dim=1)
        return grad_y, grad_w
    if op == "quantize":
        x, n = s["x"].double(), case["n"]
        if case["layout"] == "tile":
            r = x.shape[0]
            q, scales = x.new_zeros(r, -(-n // 16) * 16), x.new_zeros(-(-r // BLOCK), -(-n // BLOCK))
            for i in range(scales.shape[0]):
                rows = slice(i * BLOCK, min(r, (i + 1) * BLOCK))
                most = torch.nn.functional.pad(x[rows].abs().amax(dim=0), (0, -n % BLOCK)).view(-1, BLOCK).amax(dim=1)
                scales[i] = most.clamp(min=LEAST) / LARGEST[case["to"]]
                q[rows, :n] = _round8(x[rows] / scales[i].float().double().repeat_interleave(BLOCK)[:n], case["to"])
            return q, scales
        rows = torch.zeros(total, n, dtype=torch.float64, device="cuda")
        rows[slot] = x[token]
        if case["layout"] == "row":
            q, scales = _exact_quantize(rows, case["to"], case)
            return (torch.nn.functional.pad(q, (0, 0, 0, cap - total)),
                    torch.nn.functional.pad(scales, (0, 0, 0, cap - total)))
        q, scales = _exact_quantize(rows.t().contiguous(), case["to"], case)
        return (torch.nn.functional.pad(q, (0, s["out"].shape[1] - q.shape[1])),
                torch.nn.functional.pad(scales, (0, s["scales"].shape[1] - scales.shape[1])))
    # products: each expert's segment by itself
    def wide(q, scales, rows):
        v = q.double()
        for i in range(scales.shape[0]):
            v[i * rows:(i + 1) * rows] *= scales[i].double().repeat_interleave(BLOCK)[:v.shape[1]]
        return v
    a = s["a"].double() * s["sa"].double().repeat_interleave(BLOCK, dim=1)[:, :s["a"].shape[1]]
    if case["kind"] == "inner":
        b = s["b"].double() * s["sb"].double().repeat_interleave(BLOCK, dim=1)[:, :s["b"].shape[1]]
        out = torch.zeros(E, case["m"], case["n"], dtype=torch.float64, device="cuda")
        for e in range(E):
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            out[e] = a[:, lo:hi] @ b[:, lo:hi].t()
        return out
    of_b = BLOCK if case["b"] == "tile" else 1
    if case["kind"] == "none":
        return a @ wide(s["b"], s["sb"], of_b).t()
    out = torch.zeros(cap, case["n"], dtype=torch.float64, device="cuda")
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            out[lo:hi] = a[lo:hi] @ wide(s["b"][e], s["sb"][e], of_b).t()
    return out
