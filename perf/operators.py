"""The serving operators' cases: products with packed low-bit weights, and the norm in front of them.

A layer that the solver has rounded is stored as integer codes c (m x n, `bits` each) with fp32 scales, one a row or
one a group of `group` columns: w_ij = s_i,g(j) (c_ij - (2^bits - 1) / 2). The operators:

  matvec  y_ti = a_t sum_g s_ig sum_{j in g} x_tj (c_ij - (2^bits - 1) / 2) for T tokens, x in fp32, bf16, fp16, or in
          8 bits (int8, e4m3) with a scale a_t for each token
  norm    h = x + r, v = gain h / sqrt(mean(h^2) + eps), optionally rotated by the randomised Hadamard matrix that the
          layer's weights were rotated by; out in x's type, or in 8 bits with a scale for each token
  layer   a norm with 8-bit output and the product that reads it
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8,
          "e4m3": torch.float8_e4m3fn}
TOP = {"i8": 127.0, "e4m3": 448.0}  # what the largest magnitude of a token is scaled to
EPS = 1e-5


def listed():
    return [
        # one token of a decoding step enters a layer of hidden size 4096: all latency
        {"name": "norm_decode", "op": "norm", "T": 1, "n": 4096, "x": "bf16", "y": "bf16", "residual": True,
         "rotate": False, "pad": 0},
        # a batch of 37 decoding requests in front of a rotated layer with 14336 inputs (2^11 times 7)
        {"name": "norm_batch_rotated", "op": "norm", "T": 37, "n": 14336, "x": "f16", "y": "e4m3", "residual": True,
         "rotate": True, "pad": 0},
        # a prompt in front of a rotated layer of width 8192: memory traffic
        {"name": "norm_prompt_rotated", "op": "norm", "T": 4096, "n": 8192, "x": "bf16", "y": "e4m3",
         "residual": True, "rotate": True, "pad": 0},
        # fp32 activations of an odd width, rows of a wider buffer, no residual
        {"name": "norm_fp32_odd", "op": "norm", "T": 1001, "n": 4099, "x": "f32", "y": "f32", "residual": False,
         "rotate": False, "pad": 5},
        # one token through an attention projection: latency and 8 MB of codes
        {"name": "mv_attn_decode", "op": "matvec", "T": 1, "m": 4096, "n": 4096, "bits": 4, "group": 128,
         "x": "bf16", "y": "bf16", "pad": 0},
        # one token through a large up-projection at 2 bits with the solve's own row scales
        {"name": "mv_up_decode_2bit", "op": "matvec", "T": 1, "m": 28672, "n": 8192, "bits": 2, "group": 0,
         "x": "bf16", "y": "f32", "pad": 0},
        # one token in 8 bits through a down-projection with small groups
        {"name": "mv_down_decode_int8", "op": "matvec", "T": 1, "m": 4096, "n": 14336, "bits": 4, "group": 64,
         "x": "i8", "y": "bf16", "pad": 0},
        # a few tokens (speculative decoding), odd sizes, a partial last group, rows of a wider buffer
        {"name": "mv_ragged_fp16", "op": "matvec", "T": 7, "m": 4099, "n": 4013, "bits": 3, "group": 32,
         "x": "f16", "y": "f16", "pad": 3},
        # the framework's own fp32 activations, a batch of 16 requests
        {"name": "mv_batch_fp32", "op": "matvec", "T": 16, "m": 8192, "n": 8192, "bits": 4, "group": 128,
         "x": "f32", "y": "f32", "pad": 0},
        # a batch of 48 requests through an up-projection
        {"name": "mv_batch_bf16", "op": "matvec", "T": 48, "m": 14336, "n": 4096, "bits": 4, "group": 128,
         "x": "bf16", "y": "bf16", "pad": 0},
        # a prompt of 2048 tokens in 8 bits through an up-projection: matrix-core work
        {"name": "mv_prompt_int8", "op": "matvec", "T": 2048, "m": 14336, "n": 4096, "bits": 4, "group": 128,
         "x": "i8", "y": "bf16", "pad": 0},
        # a decoding step of four requests: norm, rotation and 8-bit rounding, then the up-projection
        {"name": "layer_decode", "op": "layer", "T": 4, "m": 14336, "n": 4096, "bits": 4, "group": 128, "x": "bf16",
         "y": "bf16", "q": "i8", "residual": True, "rotate": True, "pad": 0},
    ]


def draw(rng):
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        how = rng.random()  # most widths are multiples of 128 or of 32, some are odd
        v = v // 128 * 128 if how < 0.5 and v >= 256 else v // 32 * 32 if how < 0.75 and v >= 64 else v
        return max(lo, min(hi, v))

    def tokens(most):
        if rng.random() < 0.25:
            return 1
        return max(1, min(most, int(round(math.exp(rng.uniform(0.0, math.log(2048.0)))))))

    pad = rng.choice([0, 0, 0, 1, 8, 40])
    op = rng.choice(["norm", "matvec", "matvec", "layer"])
    if op == "norm":
        n = size(64, 16384)
        x = rng.choice(["f32", "bf16", "f16"])
        return {"op": op, "T": tokens(4096 * 8192 // n // 2), "n": n, "x": x, "y": rng.choice([x, "e4m3"]),
                "residual": rng.random() < 0.7, "rotate": rng.random() < 0.5, "pad": pad}
    m, n = size(256, 28672), size(256, 16384)
    if m * n > 28672 * 8192:
        n = 28672 * 8192 // m
    T = tokens(2048 * 14336 * 4096 // (m * n) // 4)
    bits = rng.choice([2, 3, 4, 4, 4])
    group = rng.choice([0, 32, 64, 128, 128, 256])
    if op == "layer":
        return {"op": op, "T": T, "m": m, "n": n, "bits": bits, "group": group, "x": rng.choice(["f32", "bf16"]),
                "y": "bf16", "q": rng.choice(["i8", "e4m3"]), "residual": rng.random() < 0.7,
                "rotate": rng.random() < 0.5, "pad": pad}
    return {"op": op, "T": T, "m": m, "n": n, "bits": bits, "group": group,
            "x": rng.choice(["f32", "bf16", "bf16", "f16", "i8", "e4m3"]), "y": rng.choice(["f32", "bf16", "f16"]),
            "pad": pad}


def _groups(case):
    return -(-case["n"] // case["group"]) if case["group"] else 1


def prepare(case, seed):
    """Activations with some large channels, as a transformer has them; codes as a solve leaves them."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    T, n, pad = case["T"], case["n"], case["pad"]
    st = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    x = torch.empty(T, n + pad, dtype=DTYPES[case["x"]], device=dev)[:, :n]
    act = normal(T, n) * (0.5 + normal(n).square())
    if case["op"] == "matvec" and case["x"] in TOP:
        top = TOP[case["x"]]
        st["xs"] = act.abs().amax(1) / top
        q = act / st["xs"][:, None]
        x.copy_(q.round().clamp(-top, top) if case["x"] == "i8" else q)
    else:
        x.copy_(act)
    st["x"] = x
    if case["op"] != "matvec":
        st["gain"] = (1.0 + 0.2 * normal(n)).to(x.dtype)
        st["r"] = (3.0 * normal(T, n)).to(x.dtype) if case["residual"] else None
        st["seed"] = int(seed) + 1 if case["rotate"] else None  # the seed that the layer was rotated with
    if case["op"] != "norm":
        m, top = case["m"], 2 ** case["bits"] - 1
        st["codes"] = (normal(m, n) * (top / 5.0) + top / 2.0).round_().clamp_(0, top).to(torch.uint8)
        st["scales"] = (0.02 + 0.02 * torch.rand(m, _groups(case), generator=g, device=dev)) / top
        if own:
            import kronecker_hessian_rounding_amd as bk
            st["w"] = bk.pack(st.pop("codes"), st.pop("scales"), case["bits"], case["group"])
    return st


# ------------------------------------------------------------------ plain form
def _hadamard(b, like):
    """The Sylvester matrix of order b: (-1)^popcount(i & j)."""
    i = torch.arange(b, device=like.device)
    p = i[:, None] & i
    p = p ^ (p >> 8)
    p = p ^ (p >> 4)
    p = p ^ (p >> 2)
    p = p ^ (p >> 1)
    return (1 - 2 * (p & 1)).to(like.dtype)


def _signs(seed, n, like):
    """-1 where bit 63 of SplitMix64's output i is set (int64 arithmetic wraps as uint64 does)."""
    def wrap(c):
        return c - (1 << 64) if c >> 63 else c

    def lsr(z, k):
        return (z >> k) & ((1 << (64 - k)) - 1)

    z = (torch.arange(n, device=like.device) + 1) * wrap(0x9E3779B97F4A7C15) + wrap(seed & ((1 << 64) - 1))
    z = (z ^ lsr(z, 30)) * wrap(0xBF58476D1CE4E5B9)
    z = (z ^ lsr(z, 27)) * wrap(0x94D049BB133111EB)
    z = z ^ lsr(z, 31)
    return torch.where(z < 0, -1.0, 1.0).to(like.dtype)


def _rotate(v, seed):
    """Rows of v times U^T, U = (I (x) H_b / sqrt(b)) diag(signs): H_b as the product H_p (x) H_q of two small ones."""
    T, n = v.shape
    b = n & -n
    k = b.bit_length() - 1
    p, q = 1 << (k // 2), 1 << (k - k // 2)
    z = (v * _signs(seed, n, v)).reshape(T * (n // b), p, q)
    z = torch.matmul(z.reshape(-1, q), _hadamard(q, v)).reshape(-1, p, q)
    z = torch.matmul(z.transpose(1, 2).reshape(-1, p), _hadamard(p, v)).reshape(-1, q, p).transpose(1, 2)
    return z.reshape(T, n) * b ** -0.5


def _norm(st, out):
    h = st["x"].float()
    if st["r"] is not None:
        h = h + st["r"].float()
    v = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * st["gain"].float()
    if st["seed"] is not None:
        v = _rotate(v, st["seed"])
    h = h.to(st["x"].dtype) if st["r"] is not None else None
    if out not in TOP:
        return v.to(DTYPES[out]), None, h
    s = v.abs().amax(1) / TOP[out]
    q = torch.where(s[:, None] > 0, v / s[:, None], 0.0)
    return (q.round() if out == "i8" else q).clamp(-TOP[out], TOP[out]).to(DTYPES[out]), s, h


def _matvec(x, xs, st):
    case = st["case"]
    w = st["codes"].float() - (2 ** case["bits"] - 1) / 2
    if case["group"]:
        w = w * st["scales"].repeat_interleave(case["group"], 1)[:, :case["n"]]
    else:
        w = w * st["scales"]
    y = torch.matmul(x.float(), w.t())
    return (y if xs is None else y * xs[:, None]).to(DTYPES[case["y"]])


def run(st):
    case = st["case"]
    if own:
        import kronecker_hessian_rounding_amd as bk
        if case["op"] == "matvec":
            return bk.matvec(st["x"], st["w"], x_scale=st.get("xs"), out_dtype=DTYPES[case["y"]])
        out = DTYPES[case["y"] if case["op"] == "norm" else case["q"]]
        r = bk.rmsnorm(st["x"], st["gain"], residual=st["r"], eps=EPS, rotate_seed=st["seed"], out_dtype=out)
        if case["op"] == "norm":
            return {"y": r.y, "scale": r.scale, "sum": r.sum}
        return {"y": bk.matvec(r.y, st["w"], x_scale=r.scale, out_dtype=DTYPES[case["y"]]), "sum": r.sum}
    if case["op"] == "matvec":
        return _matvec(st["x"], st.get("xs"), st)
    if case["op"] == "norm":
        y, s, h = _norm(st, case["y"])
        return {"y": y, "scale": s, "sum": h}
    q, s, h = _norm(st, case["q"])
    return {"y": _matvec(q, s, st), "sum": h}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The same outputs in 64 bits: signs from Python integers, the rotation as butterflies, the codes one group at a
    time."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    x = st["x"].double()
    T, n = x.shape
    out = {}
    xs = st["xs"].double() if "xs" in st else None
    if case["op"] != "matvec":
        if st["r"] is not None:
            x = x + st["r"].double()
            out["sum"] = x
        v = x / (x.square().sum(1, keepdim=True) / n + EPS).sqrt() * st["gain"].double()
        if st["seed"] is not None:
            with np.errstate(over="ignore"):
                z = np.uint64(st["seed"]) + np.arange(1, n + 1, dtype=np.uint64) * np.uint64(0x9E3779B97F4A7C15)
                z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
                z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
                z = z ^ (z >> np.uint64(31))
            v = v * torch.from_numpy(1.0 - 2.0 * (z >> np.uint64(63)).astype(np.float64)).to(v.device)
            h = 1
            while n % (2 * h) == 0:
                v = v.reshape(T, n // (2 * h), 2, h)
                v = (torch.stack([v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]], 2) / math.sqrt(2.0)).reshape(T, n)
                h *= 2
        kind = case["y"] if case["op"] == "norm" else case["q"]
        if kind in TOP:
            xs = v.abs().amax(1) / TOP[kind]
            v = v / xs.clamp_min(1e-300)[:, None]
            v = v.round() if kind == "i8" else v.float().to(DTYPES[kind]).double()
        if case["op"] == "norm":
            return {"y": v, "scale": xs if kind in TOP else None, "sum": out.get("sum")}
        x = v
    m, g = case["m"], case["group"] or n
    y = torch.zeros(T, m, dtype=torch.float64, device=x.device)
    for k in range(_groups(case)):
        c = st["codes"][:, k * g:(k + 1) * g].double() * 2 - (2 ** case["bits"] - 1)
        y += torch.matmul(x[:, k * g:(k + 1) * g], c.t()) * (st["scales"][:, k].double() / 2)
    out["y"] = y if xs is None else y * xs[:, None]
    if case["op"] == "matvec":
        return out["y"]
    return {"y": out["y"], "sum": out.get("sum")}


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1, "e4m3": 1}
    T, n = case["T"], case["n"]
    byts, flops = 0, 0
    if case["op"] != "matvec":
        sx = size[case["x"]]
        byts += T * n * sx * (3 if case["residual"] else 1) + n * sx
        flops += T * n * (5 + ((n & -n).bit_length() - 1 if case["rotate"] else 0))
        if case["op"] == "norm":
            byts += T * n * size[case["y"]] + (4 * T if case["y"] in TOP else 0)
    if case["op"] != "norm":
        m = case["m"]
        byts += m * n * case["bits"] // 8 + 4 * m * _groups(case) + T * m * size[case["y"]]
        flops += 2 * T * m * n
        if case["op"] == "matvec":
            byts += T * n * size[case["x"]] + (4 * T if case["x"] in TOP else 0)
    return {"bytes": byts, "flops": flops}
