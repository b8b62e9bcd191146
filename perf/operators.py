"""Cases that measure the row operators beside top-k: routing to experts with its gradient, a sampler's
probabilities (from whole logit rows and from top-k lists) and the verification of drafted tokens."""
import torch

own = False

SIZES = {"bf16": 2, "fp32": 4}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _route(name, tokens, experts, k, dtype, score, bias, groups=1, topk_groups=1, group_top=1, renorm=True,
           scale=1.0, masked=0, grad=False):
    c = {"name": name, "op": "route_grad" if grad else "route", "tokens": tokens, "experts": experts, "k": k,
         "dtype": dtype, "score": score, "bias": bias, "groups": groups, "topk_groups": topk_groups,
         "group_top": group_top, "renorm": renorm, "scale": scale, "masked": masked}
    return c


def listed():
    return [
        # one decode step of a small batch: latency
        _route("route decode 4x256", 4, 256, 8, "bf16", "sigmoid", True, 8, 4, 2, True, 2.5),
        # a prefill chunk or training micro-batch of a large router with balance bias and groups
        _route("route train 65536x256", 65536, 256, 8, "fp32", "sigmoid", True, 8, 4, 2, True, 2.5),
        # an odd number of experts and tokens, some experts switched off by their logits
        _route("route softmax 4099x61", 4099, 61, 6, "bf16", "softmax", False, masked=5),
        # the gradients of the two training routers
        _route("route grad 65536x256", 65536, 256, 8, "fp32", "sigmoid", True, 8, 4, 2, True, 2.5, grad=True),
        _route("route grad softmax 5003x128", 5003, 128, 4, "bf16", "softmax", False, renorm=False, grad=True),
        # the sampler's whole batch over its vocabulary, with a temperature for each request
        {"name": "softmax 256x129280", "op": "softmax", "rows": 256, "n": 129280, "dtype": "fp32", "out": "fp32"},
        # a few requests over a vocabulary of odd size, logits in 16 bits
        {"name": "softmax 7x50001", "op": "softmax", "rows": 7, "n": 50001, "dtype": "bf16", "out": "fp32"},
        # the sampler's lists of 512, as whole rows for the verification
        {"name": "list softmax 256x512", "op": "list_softmax", "rows": 256, "n": 129280, "k": 512, "dtype": "fp32",
         "out": "fp32", "top_p": True},
        # one request with a short list, latency
        {"name": "list softmax 1x50", "op": "list_softmax", "rows": 1, "n": 32003, "k": 50, "dtype": "bf16",
         "out": "fp32", "top_p": True},
        # one request with three drafted tokens: latency
        {"name": "verify 1x3 x 129280", "op": "verify", "batch": 1, "drafts": 3, "n": 129280, "dtype": "fp32",
         "kind": "probs"},
        # a serving batch of the sampler's size, drafts from a draft model's probabilities
        {"name": "verify 256x3 x 129280", "op": "verify", "batch": 256, "drafts": 3, "n": 129280, "dtype": "fp32",
         "kind": "probs"},
        # drafts looked up in the text (no draft probabilities), ragged draft lengths, an odd vocabulary in 16 bits
        {"name": "verify lookup 48x7 x 32003", "op": "verify", "batch": 48, "drafts": 7, "n": 32003, "dtype": "bf16",
         "kind": "tokens"},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "softmax", "list_softmax", "verify", "verify"])
    dtype = rng.choice(["bf16", "fp32"])
    if op.startswith("route"):
        groups = rng.choice([1, 1, 2, 4, 8])
        size = max(2, _log(rng, 8, 512) // groups)
        topk_groups = rng.randint(1, groups)
        k = min(size * topk_groups, rng.randint(1, 16))
        score, bias = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5
        c = _route("", _log(rng, 1, 32768), size * groups, k, dtype, score, bias, groups, topk_groups,
                   rng.choice([1, 2]), rng.random() < 0.6, rng.choice([1.0, 2.5]),
                   rng.choice([0, 0, 3]) if size * groups > 16 else 0, op == "route_grad")
        del c["name"]
        return c
    n = _log(rng, 1000, 129280)
    if op == "softmax":
        return {"op": op, "rows": min(_log(rng, 1, 256), 256 * 129280 // n), "n": n, "dtype": dtype,
                "out": rng.choice(["bf16", "fp32"])}
    if op == "list_softmax":
        return {"op": op, "rows": _log(rng, 1, 256), "n": n, "k": _log(rng, 1, 1000), "dtype": dtype,
                "out": rng.choice(["bf16", "fp32"]), "top_p": rng.random() < 0.7}
    return {"op": op, "batch": _log(rng, 1, 128), "drafts": rng.randint(0, 8), "n": n, "dtype": dtype,
            "kind": rng.choice(["probs", "tokens"])}


def _logits(g, rows, n, peak=4.0):
    """Sampler logits: a Zipf bias over the vocabulary, another order in each row, and noise."""
    rank = torch.rand(rows, n, generator=g, device="cuda").argsort(dim=1).float()
    return peak * torch.randn(rows, n, generator=g, device="cuda") - 1.1 * torch.log1p(rank)


def _probs(logits, dtype):
    return torch.softmax(logits, dim=1).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    op = case["op"]
    s = {"case": case}
    if op in ("route", "route_grad"):
        T, E, k = case["tokens"], case["experts"], case["k"]
        x = 1.2 * randn(T, E) + 0.5 * randn(E)
        if case["masked"]:
            x[:, torch.randperm(E, generator=g, device="cuda")[:case["masked"]]] = float("-inf")
        s["x"] = x.to(TYPES[case["dtype"]])
        s["bias"] = 0.1 * randn(E) if case["bias"] else None
        if op == "route_grad":
            s["idx"] = rand(T, E).argsort(dim=1)[:, :k].to(torch.int32).contiguous()
            s["idx"] = torch.where(torch.isinf(s["x"].gather(1, s["idx"].long())), -1, s["idx"])
            s["grad"] = randn(T, k)
        return s
    if op == "softmax":
        s["x"] = _logits(g, case["rows"], case["n"]).to(TYPES[case["dtype"]])
        s["t"] = 0.4 + rand(case["rows"])
        s["t"][torch.arange(case["rows"], device="cuda") % 8 == 5] = 0.0  # greedy requests
        return s
    if op == "list_softmax":
        R, n, k = case["rows"], case["n"], case["k"]
        v, i = _logits(g, R, n).to(TYPES[case["dtype"]]).sort(dim=1, descending=True, stable=True)
        s["vals"], s["idx"] = v[:, :k].contiguous(), i[:, :k].to(torch.int32).contiguous()
        s["t"] = 0.4 + rand(R)
        s["t"][torch.arange(R, device="cuda") % 8 == 5] = 0.0
        s["ks"] = torch.randint(1, k + 1, (R,), generator=g, device="cuda", dtype=torch.int32)
        s["top_p"] = 0.5 + 0.5 * rand(R) if case["top_p"] else None
        return s
    B, K, n, dt = case["batch"], case["drafts"], case["n"], TYPES[case["dtype"]]
    base = _logits(g, B * (K + 1), n, 3.0)
    target = _probs(base, dt)
    s["target"] = target.view(B, K + 1, n)
    if case["kind"] == "probs":
        q = _probs((base + 0.7 * randn(B * (K + 1), n)).view(B, K + 1, n)[:, :K].reshape(B * K, n), dt)
        s["draft"] = q.view(B, K, n)
    else:
        q, s["draft"] = torch.softmax(2 * base, dim=1).view(B, K + 1, n)[:, :K].reshape(B * K, n), None
    noise = -torch.log1p(-rand(B * K, n))
    s["tokens"] = (q.float() / noise.clamp(min=1e-30)).argmax(dim=1).to(torch.int32).view(B, K) if K else \
        torch.empty(B, 0, dtype=torch.int32, device="cuda")
    s["lens"] = torch.randint(0, K + 1, (B,), generator=g, device="cuda", dtype=torch.int32) \
        if case["kind"] == "tokens" else None
    s["accept_u"], s["sample_u"] = rand(B, K), rand(B)
    return s


def _scores(x, score):
    """The experts' scores in 64 bits; an expert whose logit is -inf has score 0."""
    x = x.double()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    m = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(m), 0, m))
    return e / e.sum(dim=1, keepdim=True).clamp(min=1e-300)


def _plain_route(s, c):
    x, T, E, k = s["x"], c["tokens"], c["experts"], c["k"]
    p = _scores(x, c["score"])
    gone = torch.isinf(x)
    # without a bias the order of the scores is that of the logits
    choice = p + s["bias"].double() if s["bias"] is not None else x.double()
    choice = torch.where(gone, float("-inf"), choice)
    if c["groups"] > 1:
        G = c["groups"]
        best = (choice if s["bias"] is not None or c["group_top"] == 1 else torch.where(gone, float("-inf"), p))
        top = best.view(T, G, E // G).sort(dim=2, descending=True)[0][:, :, :c["group_top"]]
        none = torch.isinf(top[:, :, 0])
        of_group = torch.where(none, float("-inf"), torch.where(torch.isinf(top), 0, top).sum(dim=2))
        chosen = of_group.sort(dim=1, descending=True, stable=True)[1][:, :c["topk_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, chosen, True)
        choice = torch.where(keep.repeat_interleave(E // G, dim=1), choice, float("-inf"))
    v, i = choice.sort(dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    empty = torch.isinf(v)
    w = torch.where(empty, 0, p.gather(1, i))
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, 0)
    return (c["scale"] * w).float(), torch.where(empty, -1, i).to(torch.int32)


def _plain_route_grad(s, c):
    x, idx, g = s["x"], s["idx"].long(), s["grad"]
    p = _scores(x, c["score"]).float()
    hole = idx < 0
    at = idx.clamp(min=0)
    w = torch.where(hole, 0, p.gather(1, at))
    g = c["scale"] * torch.where(hole, 0, g)
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        g = torch.where(total > 0, (g - (g * w / total).sum(dim=1, keepdim=True)) / total, 0)
    ds = torch.zeros_like(p).scatter_add_(1, at, torch.where(hole, 0, g))
    if c["score"] == "sigmoid":
        dx = ds * p * (1 - p)
    else:
        dx = p * (ds - (ds * p).sum(dim=1, keepdim=True))
    return dx.to(x.dtype)


def _plain_softmax(s, c):
    x, t = s["x"].float(), s["t"][:, None]
    m, first = x.max(dim=1, keepdim=True)[0], x.argmax(dim=1, keepdim=True)
    e = torch.exp((x - m) / torch.where(t > 0, t, 1))
    p = e / e.sum(dim=1, keepdim=True)
    hot = torch.zeros_like(x).scatter_(1, first, 1.0)
    return torch.where(t > 0, p, hot).to(TYPES[c["out"]])


def _plain_list_softmax(s, c):
    v, t = s["vals"].double(), s["t"][:, None].double()
    at = torch.arange(c["k"], device=v.device)[None]
    live = (at < s["ks"][:, None]) & ((t > 0) | (at == 0))
    e = torch.where(live, torch.exp((v - v[:, :1]) / torch.where(t > 0, t, 1)), 0)
    if s["top_p"] is not None:
        before = e.cumsum(dim=1) - e
        e = torch.where((before < s["top_p"][:, None].double() * e.sum(dim=1, keepdim=True)) | (at == 0), e, 0)
    p = (e / e.sum(dim=1, keepdim=True)).to(TYPES[c["out"]])
    return torch.zeros(c["rows"], c["n"], dtype=p.dtype, device=p.device).scatter_(1, s["idx"].long(), p)


def _plain_verify(s, c):
    target, draft, tok = s["target"], s["draft"], s["tokens"].long()
    B, K = c["batch"], c["drafts"]
    b = torch.arange(B, device=target.device)
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), K, device=target.device)
    at = torch.arange(K, device=target.device)[None]
    p = target[:, :K].gather(2, tok[:, :, None])[:, :, 0].double()
    q = draft.gather(2, tok[:, :, None])[:, :, 0].double() if draft is not None else torch.ones_like(p)
    taken = ((s["accept_u"].double() * q < p) & (at < lens[:, None])).long().cumprod(dim=1)
    got = taken.sum(dim=1)
    refused = got < lens
    rest = target[b, got].double()
    whole = rest
    if K:
        r = got.clamp(max=K - 1)
        if draft is not None:
            less = draft[b, r].double()
        else:
            less = torch.zeros_like(rest).scatter_(1, tok[b, r][:, None], float("inf"))
        rest = torch.where(refused[:, None], (rest - less).clamp(min=0), rest)
        rest = torch.where(rest.sum(dim=1, keepdim=True) > 0, rest, whole)
    run_sum = rest.cumsum(dim=1)
    total = run_sum[:, -1:]
    token = (run_sum <= s["sample_u"].double()[:, None] * total).sum(dim=1)
    token = torch.where(total[:, 0] > 0, token.clamp(max=c["n"] - 1), -1)
    out = torch.full((B, K + 1), -1, dtype=torch.int32, device=target.device)
    out[:, :K] = torch.where(taken > 0, s["tokens"], -1)
    out.scatter_(1, got[:, None], token.to(torch.int32)[:, None])
    return out, got.to(torch.int32)


def _own(s, c):
    import top_selection_amd as ts
    op = c["op"]
    if op in ("route", "route_grad"):
        score = ts.SCORE_SIGMOID if c["score"] == "sigmoid" else ts.SCORE_SOFTMAX
        if op == "route":
            return ts.ds_route(s["x"], c["k"], bias=s["bias"], score=score, groups=c["groups"],
                               topk_groups=c["topk_groups"], group_top=c["group_top"], renormalize=c["renorm"],
                               scale=c["scale"])
        return ts.ds_route_grad(s["x"], s["idx"], s["grad"], score=score, renormalize=c["renorm"], scale=c["scale"])
    if op == "softmax":
        return ts.ds_softmax(s["x"], temperature=s["t"], out_dtype=TYPES[c["out"]])
    if op == "list_softmax":
        return ts.ds_topk_softmax(s["vals"], s["idx"], c["n"], ks=s["ks"], temperature=s["t"], top_p=s["top_p"],
                                  out_dtype=TYPES[c["out"]])
    return ts.ds_verify(s["target"], s["draft"], s["tokens"], s["accept_u"], s["sample_u"], draft_lens=s["lens"])


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return {"route": _plain_route, "route_grad": _plain_route_grad, "softmax": _plain_softmax,
            "list_softmax": _plain_list_softmax, "verify": _plain_verify}[c["op"]](state, c)


def work(case):
    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, k, b = case["tokens"], case["experts"], case["k"], SIZES[case["dtype"]]
        if op == "route":
            return {"bytes": T * E * b + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": T * E * 6}
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": T * E * b * (2 if dense else 1) + T * k * (8 if dense else 8 + b), "flops": T * E * 6}
    if op == "softmax":
        return {"bytes": case["rows"] * case["n"] * (SIZES[case["dtype"]] + SIZES[case["out"]]) + 4 * case["rows"],
                "flops": case["rows"] * case["n"] * 5}
    if op == "list_softmax":
        return {"bytes": case["rows"] * (case["k"] * (SIZES[case["dtype"]] + 4) + case["n"] * SIZES[case["out"]] + 12),
                "flops": case["rows"] * case["k"] * 6}
    B, K, n, b = case["batch"], case["drafts"], case["n"], SIZES[case["dtype"]]
    # a row of the target for each sequence; about half of the sequences refuse a draft and read its row too
    rows = 1.5 if case["kind"] == "probs" and K else 1.0
    return {"bytes": int(B * n * b * rows) + B * (K + 2) * 4 + B * K * (8 + 2 * b) + 4 * B, "flops": int(B * n * 3)}


def exact(case, seed):
    """The operators' definitions in 64 bits, row by row in numpy."""
    import numpy as np
    s = prepare(case, seed)
    a = {k: (v.double() if v.is_floating_point() else v).cpu().numpy() for k, v in s.items()
         if isinstance(v, torch.Tensor)}
    op = case["op"]
    if op in ("route", "route_grad"):
        x = a["x"]
        with np.errstate(over="ignore"):
            if case["score"] == "sigmoid":
                p = 0.5 * (1 + np.tanh(x / 2))
            else:
                p = np.exp(x - np.logaddexp.reduce(x, axis=1)[:, None])
        T, E = x.shape
        if op == "route_grad":
            at = a["idx"]
            hit = np.zeros((T, E))
            g = np.zeros((T, E))
            rows, cols = np.nonzero(at >= 0)
            hit[rows, at[rows, cols]] = 1
            g[rows, at[rows, cols]] = a["grad"][rows, cols] * case["scale"]
            if case["renorm"]:
                S = (hit * p).sum(axis=1, keepdims=True)
                S[S == 0] = np.inf
                g = hit * (g / S - (g * p).sum(axis=1, keepdims=True) / S ** 2)
            d = g * p * (1 - p) if case["score"] == "sigmoid" else p * g - p * (g * p).sum(axis=1, keepdims=True)
            return d
        c = np.where(np.isinf(x), -np.inf, p + a["bias"] if case["bias"] else x)
        G = case["groups"]
        if G > 1:
            byg = np.sort((c if case["bias"] or case["group_top"] == 1 else np.where(np.isinf(x), -np.inf, p))
                          .reshape(T, G, E // G), axis=2)[:, :, ::-1][:, :, :case["group_top"]]
            score = np.where(np.isinf(byg[:, :, 0]), -np.inf, np.where(np.isinf(byg), 0, byg).sum(axis=2))
            rank = np.argsort(np.argsort(-score, axis=1, kind="stable"), axis=1, kind="stable")
            c = np.where(np.repeat(rank < case["topk_groups"], E // G, axis=1), c, -np.inf)
        i = np.argsort(-c, axis=1, kind="stable")[:, :case["k"]]
        empty = np.isinf(np.take_along_axis(c, i, 1))
        w = np.where(empty, 0, np.take_along_axis(p, i, 1))
        if case["renorm"]:
            w = w / np.maximum(w.sum(axis=1, keepdims=True), 1e-300)
        return w * case["scale"], np.where(empty, -1, i).astype(np.int32)
    if op == "softmax":
        out = np.zeros(a["x"].shape)
        for r, (x, t) in enumerate(zip(a["x"], a["t"])):
            if t > 0:
                out[r] = np.exp((x - x.max()) / t)
                out[r] /= out[r].sum()
            else:
                out[r, int(np.argmax(x))] = 1
        return out
    if op == "list_softmax":
        out = np.zeros((case["rows"], case["n"]))
        for r in range(case["rows"]):
            m = int(a["ks"][r]) if a["t"][r] > 0 else 1
            e = np.exp((a["vals"][r, :m] - a["vals"][r, 0]) / (a["t"][r] if a["t"][r] > 0 else 1))
            if case["top_p"]:
                e = e[:max(1, int(np.searchsorted(np.cumsum(e), a["top_p"][r] * e.sum(), side="left")) + 1)]
            out[r, a["idx"][r, :len(e)]] = e / e.sum()
        return out
    B, K = case["batch"], case["drafts"]
    out, got = np.full((B, K + 1), -1, np.int32), np.zeros(B, np.int32)
    for r in range(B):
        m, j = int(a["lens"][r]) if "lens" in a else K, 0
        while j < m:
            t = a["tokens"][r, j]
            if not a["accept_u"][r, j] * (a["draft"][r, j, t] if "draft" in a else 1.0) < a["target"][r, j, t]:
                break
            out[r, j] = t
            j += 1
        p = a["target"][r, j].copy()
        if j < m:
            rest = p - a["draft"][r, j] if "draft" in a else p.copy()
            rest[rest < 0] = 0
            if "draft" not in a:
                rest[a["tokens"][r, j]] = 0
            p = rest if rest.sum() > 0 else p
        run_sum = np.cumsum(p)
        if run_sum[-1] > 0:
            out[r, j] = int(np.searchsorted(run_sum, a["sample_u"][r] * run_sum[-1], side="right"))
        got[r] = j
    return out, got
