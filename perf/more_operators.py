"""More serving operators' cases: products in which each token names its own weights, and norms of heads.

Beside a layer that the solver has rounded (integer codes with fp32 scales, w_ij = s_i,g(j) (c_ij - (2^bits - 1) / 2)):

  lora     y_t = base_t + s_a B_a (A_a x_t), a the adapter of token t's request (or none), beside a shared projection
  route    the k experts of each token from a router's logits: softmax, or sigmoid with a bias for the choice alone
  experts  y_t = sum_j w_tj D_e (act(G_e x_t) * (U_e x_t)), e = ids_tj: the products of rounded experts (their three
           matrices as codes), from given ids or behind `route` ("moe")
  heads    v = gain h / sqrt(mean(h^2) + eps) for each head of the queries and keys, then pairs of v rotated by the
           angles position * freq
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8,
          "e4m3": torch.float8_e4m3fn}
TOP = {"i8": 127.0, "e4m3": 448.0}  # what the largest magnitude of a token is scaled to
EPS = 1e-6


def listed():
    return [
        # one request's token beside an attention projection: all latency
        {"name": "lora_decode", "op": "lora", "T": 1, "n": 4096, "m": 4096, "r": 16, "R": 8, "x": "bf16", "w": "bf16",
         "y": "bf16", "base": True, "runs": 1, "none": 0.0, "pad": 0},
        # a decoding step of 64 requests with some 48 adapters beside an up-projection, some requests without one
        {"name": "lora_batch", "op": "lora", "T": 64, "n": 4096, "m": 14336, "r": 16, "R": 48, "x": "bf16",
         "w": "bf16", "y": "bf16", "base": True, "runs": 1, "none": 0.1, "pad": 0},
        # fp32 tokens, odd sizes, an odd rank, no base, rows of a wider buffer
        {"name": "lora_fp32_odd", "op": "lora", "T": 77, "n": 4013, "m": 1027, "r": 13, "R": 6, "x": "f32", "w": "f32",
         "y": "f32", "base": False, "runs": 5, "none": 0.1, "pad": 3},
        # prompts of six requests (runs of tokens with one adapter): memory traffic
        {"name": "lora_prompt", "op": "lora", "T": 4096, "n": 4096, "m": 14336, "r": 64, "R": 6, "x": "bf16",
         "w": "bf16", "y": "bf16", "base": True, "runs": 683, "none": 0.0, "pad": 0},
        # one token's 8 of 128 experts: all latency
        {"name": "route_decode", "op": "route", "T": 1, "E": 128, "k": 8, "l": "f32", "scoring": "softmax",
         "renorm": True, "scale": 1.0, "pad": 0},
        # a prompt's 8 of 256 experts, sigmoid scores, a bias that balances the choice
        {"name": "route_prompt", "op": "route", "T": 8192, "E": 256, "k": 8, "l": "bf16", "scoring": "sigmoid",
         "renorm": True, "scale": 2.5, "pad": 0},
        # one token through many small experts, router's choice included: latency and 26 MB of codes
        {"name": "moe_decode", "op": "moe", "T": 1, "n": 2048, "I": 1408, "E": 64, "k": 6, "bits": 4, "group": 128,
         "dbits": 4, "dgroup": 128, "x": "bf16", "y": "bf16", "act": "silu", "none": 0.0, "pad": 0},
        # a batch of 16 requests through 8 large experts: nearly all of their 0.7 GB
        {"name": "moe_batch", "op": "experts", "T": 16, "n": 4096, "I": 14336, "E": 8, "k": 2, "bits": 4, "group": 128,
         "dbits": 4, "dgroup": 128, "x": "bf16", "y": "bf16", "act": "silu", "none": 0.0, "pad": 0},
        # odd sizes, fp32 tokens, codes of other widths with row scales behind the activation, a padded batch
        {"name": "moe_fp32_odd", "op": "experts", "T": 7, "n": 1003, "I": 717, "E": 5, "k": 3, "bits": 3, "group": 32,
         "dbits": 2, "dgroup": 0, "x": "f32", "y": "f32", "act": "gelu", "none": 0.3, "pad": 5},
        # a prompt in 8 bits, 64 tokens an expert on average: matrix-core work
        {"name": "moe_prompt", "op": "moe", "T": 512, "n": 2048, "I": 1408, "E": 32, "k": 4, "bits": 4, "group": 128,
         "dbits": 4, "dgroup": 128, "x": "i8", "y": "bf16", "act": "silu", "none": 0.0, "pad": 0},
        # a decoding step of four requests behind a fused projection's rows: all latency
        {"name": "heads_decode", "op": "heads", "T": 4, "hq": 32, "hk": 8, "d": 128, "rot": 128, "x": "bf16",
         "pairs": "half", "norm": True, "gain": "x", "far": 131072, "pad": 1024},
        # a prompt: memory traffic
        {"name": "heads_prompt", "op": "heads", "T": 8192, "hq": 32, "hk": 8, "d": 128, "rot": 128, "x": "bf16",
         "pairs": "half", "norm": True, "gain": "x", "far": 8192, "pad": 1024},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    def size(lo, hi):
        v = log(lo, hi)
        how = rng.random()  # most widths are multiples of 128 or of 32, some are odd
        v = v // 128 * 128 if how < 0.5 and v >= 256 else v // 32 * 32 if how < 0.75 and v >= 64 else v
        return max(lo, min(hi, v))

    pad = rng.choice([0, 0, 0, 1, 8, 40])
    op = rng.choice(["lora", "lora", "route", "experts", "moe", "experts", "heads"])
    if op == "lora":
        n, m, r = size(64, 16384), size(64, 28672), rng.choice([1, 4, 8, 8, 13, 16, 16, 16, 24, 32, 64, 100, 128])
        x = rng.choice(["f32", "f16", "bf16", "bf16", "i8", "e4m3"])
        w = rng.choice(["f16", "bf16"]) if x in TOP else x
        T = min(log(1, 4096), 4096 * 18432 * 64 // ((n + m) * r), 4096 * 18432 // (2 * (n + m)))
        T = 1 if rng.random() < 0.2 else max(1, T)
        R = min(log(1, 64), max(1, 2 ** 27 // ((n + m) * r)))
        return {"op": op, "T": T, "n": n, "m": m, "r": r, "R": R, "x": x, "w": w, "y": rng.choice(["f32", "bf16", "f16"]),
                "base": rng.random() < 0.7, "runs": log(1, max(1, T // 2)), "none": rng.choice([0.0, 0.1, 0.5]), "pad": pad}
    if op == "route":
        E = rng.choice([4, 8, 16, 32, 60, 64, 64, 128, 160, 256, 512, log(2, 512)])
        return {"op": op, "T": 1 if rng.random() < 0.2 else min(log(1, 8192), 8192 * 256 // E), "E": E,
                "k": rng.choice([k for k in (1, 2, 4, 6, 8, 8, 10, 16) if k <= E]), "l": rng.choice(["f32", "f32", "bf16", "f16"]),
                "scoring": rng.choice(["softmax", "softmax", "sigmoid"]), "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5]), "pad": pad}
    if op == "heads":
        d = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256, 2 * log(8, 128)])
        hq, hk = rng.choice([(32, 8), (32, 32), (64, 8), (16, 2), (8, 1), (28, 4), (5, 5), (12, 0)])
        T = min(log(1, 8192), 8192 * 40 * 128 // ((hq + hk) * d) // 2)
        return {"op": op, "T": max(1, T), "hq": hq, "hk": hk, "d": d,
                "rot": rng.choice([d, d, d, d // 4 * 2, 0]), "x": rng.choice(["f32", "f16", "bf16", "bf16"]),
                "pairs": rng.choice(["half", "half", "interleaved"]), "norm": rng.random() < 0.75,
                "gain": rng.choice(["x", "f32", ""]), "far": rng.choice([4096, 131072, 1048576]), "pad": pad}
    n, I = size(256, 8192), size(128, 14336)
    E = min(rng.choice([2, 4, 5, 8, 16, 32, 60, 64, 128]), max(2, 8 * 14336 * 4096 // (n * I)))
    k = rng.choice([k for k in (1, 2, 2, 4, 6, 8) if k <= E])
    T = 1 if rng.random() < 0.25 else max(1, min(log(1, 512), 512 * 4 * 2048 * 1408 // (k * n * I)))
    return {"op": op, "T": T, "n": n, "I": I, "E": E, "k": k, "bits": rng.choice([2, 3, 4, 4, 4]),
            "group": rng.choice([0, 32, 64, 128, 128, 256]), "dbits": rng.choice([2, 3, 4, 4, 4]),
            "dgroup": rng.choice([0, 32, 64, 128, 128, 256]), "x": rng.choice(["f32", "bf16", "bf16", "f16", "i8", "e4m3"]),
            "y": rng.choice(["f32", "bf16", "f16"]), "act": rng.choice(["silu", "silu", "gelu"]),
            "none": rng.choice([0.0, 0.0, 0.2]) if op == "experts" else 0.0, "pad": pad}


# ------------------------------------------------------------------ inputs
def _tokens(st, case, T, n, normal):
    """Activations with some large channels, as a transformer has them, in 8 bits with a scale for each token."""
    x = torch.empty(T, n + case["pad"], dtype=DTYPES[case["x"]], device="cuda")[:, :n]
    act = normal(T, n) * (0.5 + 0.5 * normal(n).square())
    if case["x"] in TOP:
        top = TOP[case["x"]]
        st["xs"] = act.abs().amax(1) / top
        q = act / st["xs"][:, None]
        x.copy_(q.round().clamp(-top, top) if case["x"] == "i8" else q)
    else:
        x.copy_(act)
    st["x"] = x


def _ngroups(n, group):
    return -(-n // group) if group else 1


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    st = {"case": case}
    T = case["T"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["op"] == "lora":
        n, m, r, R = case["n"], case["m"], case["r"], case["R"]
        _tokens(st, case, T, n, normal)
        wt = DTYPES[case["w"]]
        st["a"] = (normal(R, r, n) * n ** -0.5).to(wt)
        st["b"] = (normal(R, m, r) * r ** -0.5).to(wt)
        st["s"] = 0.5 + 1.5 * torch.rand(R, generator=g, device=dev)
        # requests one behind the other, `runs` tokens each; a share of them has no adapter
        req = -(-T // case["runs"])
        ids = torch.randint(0, R, (req,), generator=g, device=dev)
        ids = torch.where(torch.rand(req, generator=g, device=dev) < case["none"], -1, ids)
        st["ids"] = ids.repeat_interleave(case["runs"])[:T].to(torch.int32)
        if case["base"]:
            st["base"] = torch.empty(T, m + case["pad"], dtype=DTYPES[case["y"]], device=dev)[:, :m]
            st["base"].copy_(normal(T, m))
        return st
    if case["op"] == "heads":
        hq, hk, d = case["hq"], case["hk"], case["d"]
        # the rows of a fused projection: queries, keys, and behind them the values (pad)
        rows = torch.empty(T, (hq + hk) * d + case["pad"], dtype=DTYPES[case["x"]], device=dev)
        rows.copy_(normal(T, rows.shape[1]) * (0.3 + normal(rows.shape[1]).square()))
        st["q"] = rows[:, :hq * d].unflatten(1, (hq, d))
        st["k"] = rows[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)) if hk else None
        gt = {"x": rows.dtype, "f32": torch.float32, "": None}[case["gain"]]
        st["gq"] = (1.0 + 0.2 * normal(d)).to(gt) if gt and case["norm"] else None
        st["gk"] = (1.0 + 0.2 * normal(d)).to(gt) if gt and case["norm"] and hk else None
        rot = case["rot"]
        st["freq"] = 10000.0 ** (-torch.arange(rot // 2, device=dev, dtype=torch.float32) / max(1, rot // 2)) if rot else None
        first = torch.randint(0, case["far"], (1,), generator=g, device=dev)
        st["pos"] = (first + torch.arange(T, device=dev)) % case["far"] if rot else None
        return st
    # the router's logits: some experts are more popular than others
    E, k = case["E"], case["k"]
    lt = DTYPES[case.get("l", "f32")]
    logits = torch.empty(T, E + case["pad"], dtype=lt, device=dev)[:, :E]
    logits.copy_(normal(T, E) * 1.5 + 0.5 * normal(E))
    if case["op"] != "experts":
        st["logits"] = logits
        st["bias"] = 0.1 * normal(E) if case.get("scoring") == "sigmoid" else None
    else:
        top = torch.sort(logits.float(), dim=1, descending=True, stable=True)
        ids = top.indices[:, :k].to(torch.int32)
        # a batch that is padded: rows behind the last request name no expert
        st["ids"] = torch.where(torch.arange(T, device=dev)[:, None] < T - int(T * case["none"]), ids, -1)
        st["weights"] = torch.softmax(top.values[:, :k], 1)
    if case["op"] == "route":
        return st
    n, I = case["n"], case["I"]
    _tokens(st, case, T, n, normal)
    if own:
        import kronecker_hessian_rounding_amd as bk
    for name, m, cols, bits, group in (("gate", I, n, case["bits"], case["group"]), ("up", I, n, case["bits"], case["group"]),
                                       ("down", n, I, case["dbits"], case["dgroup"])):
        top = 2 ** bits - 1
        codes = torch.empty(E, m, cols, dtype=torch.uint8, device=dev)
        for e in range(E):
            codes[e] = (normal(m, cols) * (top / 5.0) + top / 2.0).round_().clamp_(0, top)
        ng = _ngroups(cols, group)
        scales = (0.5 + torch.rand(E, m, ng, generator=g, device=dev)) * (5.0 / top * cols ** -0.5)
        st[name] = bk.pack_experts(codes, scales, bits, group) if own else (codes, scales)
    return st


# ------------------------------------------------------------------ plain form
def _lora(st):
    case = st["case"]
    x = st["x"].float()
    y = torch.zeros(case["T"], case["m"], device=x.device)
    if st.get("base") is not None:
        y += st["base"].float()
    ids = st["ids"]
    for a in range(case["R"]):
        rows = (ids == a).nonzero()[:, 0]
        if rows.numel() == 0:
            continue
        u = torch.matmul(x[rows], st["a"][a].float().t())
        if "xs" in st:
            u = u * st["xs"][rows, None]
        y[rows] += torch.matmul(u, st["b"][a].float().t()) * st["s"][a]
    return y.to(DTYPES[case["y"]])


def _route(st):
    case = st["case"]
    if case.get("scoring", "softmax") == "sigmoid":
        # in 64 bits: sigmoids close to one another, beside a bias, decide which expert is chosen
        score = 1.0 / (1.0 + torch.exp(-st["logits"].double()))
        choice = score + st["bias"].double()
    else:
        l = st["logits"].float()
        score = torch.exp(l - l.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
        choice = l
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :case["k"]]
    w = torch.gather(score, 1, ids)
    if case.get("renorm", True):
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), (w * case.get("scale", 1.0)).float()


def _dense(pair, e, bits, group):
    codes, scales = pair[0][e], pair[1][e]
    w = codes.float() - (2 ** bits - 1) / 2
    return w * (scales.repeat_interleave(group, 1)[:, :w.shape[1]] if group else scales)


def _act(v, kind):
    if kind == "silu":
        return v / (1.0 + torch.exp(-v))
    return 0.5 * v * (1.0 + torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v)))


def _experts(st, ids, weights):
    case = st["case"]
    x = st["x"].float()
    if "xs" in st:
        x = x * st["xs"][:, None]
    y = torch.zeros(case["T"], case["n"], device=x.device)
    for e in range(case["E"]):
        hit = ids == e
        rows = hit.any(1).nonzero()[:, 0]
        if rows.numel() == 0:
            continue
        w = (weights * hit)[rows].sum(1, keepdim=True)
        h = _act(torch.matmul(x[rows], _dense(st["gate"], e, case["bits"], case["group"]).t()), case["act"])
        h = h * torch.matmul(x[rows], _dense(st["up"], e, case["bits"], case["group"]).t())
        y[rows] += w * torch.matmul(h, _dense(st["down"], e, case["dbits"], case["dgroup"]).t())
    return y.to(DTYPES[case["y"]])


def _head(h, gain, st):
    case = st["case"]
    v = h.float()
    if case["norm"]:
        v = v * torch.rsqrt(v.square().mean(2, keepdim=True) + EPS)
        if gain is not None:
            v = v * gain.float()
    rot = case["rot"]
    if rot:
        angle = st["pos"].double()[:, None] * st["freq"].double()
        c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        out = v.clone()
        if case["pairs"] == "half":
            a, b = v[..., :rot // 2], v[..., rot // 2:rot]
            out[..., :rot // 2], out[..., rot // 2:rot] = a * c - b * s, b * c + a * s
        else:
            a, b = v[..., :rot:2], v[..., 1:rot:2]
            out[..., :rot:2], out[..., 1:rot:2] = a * c - b * s, b * c + a * s
        v = out
    return v.to(h.dtype)


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import kronecker_hessian_rounding_amd as bk
        if op == "lora":
            return bk.lora(st["x"], st["a"], st["b"], st["ids"], base=st.get("base"), scales=st["s"],
                           x_scale=st.get("xs"), out_dtype=DTYPES[case["y"]])
        if op == "heads":
            return bk.head_norm(st["q"], st["k"], q_gain=st["gq"], k_gain=st["gk"], positions=st["pos"],
                                freq=st["freq"], eps=EPS, norm=case["norm"], pairs=case["pairs"])
        if op == "route":
            return bk.route(st["logits"], case["k"], scoring=case["scoring"], bias=st["bias"],
                            renormalize=case["renorm"], scale=case["scale"])
        ids, w = bk.route(st["logits"], case["k"]) if op == "moe" else (st["ids"], st["weights"])
        y = bk.experts(st["x"], st["gate"], st["up"], st["down"], ids, w, x_scale=st.get("xs"), act=case["act"],
                       out_dtype=DTYPES[case["y"]])
        return {"y": y, "ids": ids, "weights": w} if op == "moe" else y
    if op == "lora":
        return _lora(st)
    if op == "heads":
        return _head(st["q"], st["gq"], st), None if st["k"] is None else _head(st["k"], st["gk"], st)
    if op == "route":
        return _route(st)
    ids, w = _route(st) if op == "moe" else (st["ids"], st["weights"])
    y = _experts(st, ids, w)
    return {"y": y, "ids": ids, "weights": w} if op == "moe" else y


# ------------------------------------------------------------------ 64 bits
def _select(key, k):
    """The k largest, one after the other, the lowest index first among equals."""
    key = key.clone()
    out = []
    for _ in range(k):
        at = (key == key.amax(1, keepdim=True)).to(torch.uint8).argmax(1, keepdim=True)
        out.append(at)
        key.scatter_(1, at, -math.inf)
    return torch.cat(out, 1)


def exact(case, seed):
    """The same outputs in 64 bits, token by token's choice: heads as complex numbers, the codes one group at a time."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op, T = case["op"], case["T"]
    if op == "heads":
        res = []
        for h, gain in ((st["q"], st["gq"]), (st["k"], st["gk"])):
            if h is None:
                res.append(None)
                continue
            v = h.double()
            if case["norm"]:
                v = v / (v.pow(2).sum(2, keepdim=True) / case["d"] + EPS).sqrt()
                v = v if gain is None else v * gain.double()
            rot = case["rot"]
            if rot:
                z = v[..., :rot].unflatten(2, (2, rot // 2) if case["pairs"] == "half" else (rot // 2, 2))
                z = z.transpose(2, 3) if case["pairs"] == "half" else z
                z = torch.view_as_complex(z.contiguous())
                turn = st["pos"].double()[:, None, None] * st["freq"].double()
                z = torch.view_as_real(z * torch.polar(torch.ones_like(turn), turn))
                z = (z.transpose(2, 3) if case["pairs"] == "half" else z).flatten(2)
                v = torch.cat([z, v[..., rot:]], 2)
            res.append(v)
        return tuple(res)
    if op == "lora":
        x, ids = st["x"].double(), st["ids"].long()
        y = torch.zeros(T, case["m"], dtype=torch.float64, device=x.device) if st.get("base") is None else st["base"].double()
        for a in ids.unique().tolist():
            if a >= 0:
                at = ids == a
                f = st["s"][a].double() * (st["xs"][at].double() if "xs" in st else 1.0)
                u = (st["a"][a].double() @ x[at].t()) * f
                y[at] = y[at] + (st["b"][a].double() @ u).t()
        return y
    if op == "experts":
        ids, w = st["ids"].long(), st["weights"].double()
    else:
        l = st["logits"].double()
        if case.get("scoring", "softmax") == "sigmoid":
            score = torch.sigmoid(l)
            ids = _select(score + st["bias"].double(), case["k"])
        else:
            score = torch.softmax(l, 1)
            ids = _select(l, case["k"])
        w = score.gather(1, ids)
        w = (w / w.sum(1, keepdim=True) if case.get("renorm", True) else w) * case.get("scale", 1.0)
        if op == "route":
            return ids.to(torch.int32), w
    x = st["x"].double() * (st["xs"].double()[:, None] if "xs" in st else 1.0)

    def product(v, pair, e, bits, group):
        codes, scales = pair[0][e], pair[1][e]
        cols = group or codes.shape[1]
        out = 0.0
        for q in range(scales.shape[1]):
            c = codes[:, q * cols:(q + 1) * cols].double() * 2 - (2 ** bits - 1)
            out = out + (v[:, q * cols:(q + 1) * cols] @ c.t()) * (scales[:, q].double() / 2)
        return out

    y = torch.zeros(T, case["n"], dtype=torch.float64, device=x.device)
    for j in range(case["k"]):
        for e in ids[:, j].unique().tolist():
            if e >= 0:
                at = ids[:, j] == e
                v = product(x[at], st["gate"], e, case["bits"], case["group"])
                v = v * torch.sigmoid(v) if case["act"] == "silu" else \
                    v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
                v = v * product(x[at], st["up"], e, case["bits"], case["group"])
                y[at] += w[at, j, None] * product(v, st["down"], e, case["dbits"], case["dgroup"])
    return {"y": y, "ids": ids.to(torch.int32), "weights": w} if op == "moe" else y


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1, "e4m3": 1}
    T, op = case["T"], case["op"]
    if op == "heads":
        e = T * (case["hq"] + case["hk"]) * case["d"]
        return {"bytes": 2 * e * size[case["x"]] + 8 * T, "flops": e * (4 * case["norm"] + 3 * bool(case["rot"]))}
    if op == "route":
        return {"bytes": T * case["E"] * size[case["l"]] + 8 * T * case["k"], "flops": 4 * T * case["E"]}
    n = case["n"]
    tok = T * n * size[case["x"]] + (4 * T if case["x"] in TOP else 0)
    if op == "lora":
        m, r = case["m"], case["r"]
        req = -(-T // case["runs"])
        used = case["R"] * (1.0 - (1.0 - (1.0 - case["none"]) / case["R"]) ** req)  # adapters named, on average
        return {"bytes": int(tok + used * r * (n + m) * size[case["w"]] + T * m * size[case["y"]] * (1 + case["base"])),
                "flops": int(2 * T * (1.0 - case["none"]) * r * (n + m))}
    I, E, k = case["I"], case["E"], case["k"]
    live = T - int(T * case["none"])
    used = E * (1.0 - (1.0 - k / E) ** live)  # experts named, on average
    each = 2 * (I * n * case["bits"] // 8 + 4 * I * _ngroups(n, case["group"])) + \
        n * I * case["dbits"] // 8 + 4 * n * _ngroups(I, case["dgroup"])
    return {"bytes": int(tok + used * each + T * n * size[case["y"]] + 8 * T * k + (4 * T * E if op == "moe" else 0)),
            "flops": 6 * live * k * n * I}
