"""What is measured of the decode layer's operators around the ternary products.

Four operators: the ternary product with bias, activation and residual in its epilogue
(op "linear"), rotary positions (op "rope"), rotary positions with the append to a paged
key/value cache (op "append"), and the attention of one new token over that cache (op
"attend").  The head layout 40 query heads, 8 key/value heads, head dim 128 is the one
whose qkv projection has the 7168 rows of the 27B-class shapes.

Where `own` is false, run() computes the plain forms below; where it is true, it makes the
library's calls on the same inputs.
"""
import functools
import math

import torch

own = False

FMT = {"ptq1": 1, "pq2": 2, "q1": 3, "pq2g64": 4}
ACT = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
LAYOUT = {"half": 0, "interleaved": 1}
KV = {"f16": 0, "e4m3": 1}


def listed():
    return [
        # one decoded token through the o projection, added to the residual stream
        {"name": "linear o M1 pq2", "op": "linear", "M": 1, "N": 5120, "K": 5120, "fmt": "pq2", "bias": False,
         "act": "none", "residual": True},
        # four decoded tokens through a qkv projection with biases, the compact packing
        {"name": "linear qkv M4 ptq1", "op": "linear", "M": 4, "N": 7168, "K": 5120, "fmt": "ptq1", "bias": True,
         "act": "none", "residual": False},
        # a short prompt through a small layer with an odd number of outputs, bias and GELU
        {"name": "linear M100 odd q1 gelu", "op": "linear", "M": 100, "N": 1001, "K": 1024, "fmt": "q1", "bias": True,
         "act": "gelu", "residual": False},
        # a prompt through the down projection, added to the residual stream
        {"name": "linear down M2048 pq2", "op": "linear", "M": 2048, "N": 5120, "K": 17408, "fmt": "pq2",
         "bias": False, "act": "none", "residual": True},
        # one decoded token: its query and key heads rotated, far into a long context
        {"name": "rope T1", "op": "rope", "T": 1, "heads": 48, "dim": 128, "rotary": 128, "layout": "half",
         "scaling": "plain", "span": 262144},
        # a prompt of odd length, pairs next to each other
        {"name": "rope T8191", "op": "rope", "T": 8191, "heads": 48, "dim": 128, "rotary": 128,
         "layout": "interleaved", "scaling": "plain", "span": 262144},
        # a decode batch into an 8-bit cache
        {"name": "append T32 e4m3", "op": "append", "T": 32, "q_heads": 40, "kv_heads": 8, "dim": 128, "rotary": 128,
         "layout": "half", "scaling": "plain", "span": 32768, "page": 16, "kv": "e4m3"},
        # a prompt into a 16-bit cache, half of each head rotated, frequencies stretched for a long context
        {"name": "append T4096 f16", "op": "append", "T": 4096, "q_heads": 40, "kv_heads": 8, "dim": 128,
         "rotary": 64, "layout": "half", "scaling": "yarn", "span": 131072, "page": 64, "kv": "f16"},
        # one sequence early in its answer
        {"name": "attend B1 L333", "op": "attend", "B": 1, "q_heads": 40, "kv_heads": 8, "dim": 128, "page": 16,
         "kv": "f16", "min_len": 333, "max_len": 333, "window": 0},
        # one sequence with a long context
        {"name": "attend B1 L131072", "op": "attend", "B": 1, "q_heads": 40, "kv_heads": 8, "dim": 128, "page": 64,
         "kv": "f16", "min_len": 131072, "max_len": 131072, "window": 0},
        # a serving batch of ragged lengths
        {"name": "attend B64 ragged f16", "op": "attend", "B": 64, "q_heads": 40, "kv_heads": 8, "dim": 128,
         "page": 16, "kv": "f16", "min_len": 64, "max_len": 8192, "window": 0},
        # a serving batch on an 8-bit cache, longer and more ragged
        {"name": "attend B64 ragged e4m3", "op": "attend", "B": 64, "q_heads": 40, "kv_heads": 8, "dim": 128,
         "page": 32, "kv": "e4m3", "min_len": 256, "max_len": 16384, "window": 0},
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "rope", "append", "attend", "attend"])
    if op == "linear":
        return {"op": op, "M": _log(rng, 1, 2048), "N": _log(rng, 64, 5120), "K": 128 * _log(rng, 1, 136),
                "fmt": rng.choice(sorted(FMT)), "bias": rng.random() < 0.5, "act": rng.choice(sorted(ACT)),
                "residual": rng.random() < 0.5}
    dim = rng.choice([64, 128, 128, 256])
    if op == "rope":
        return {"op": op, "T": _log(rng, 1, 8192), "heads": rng.randint(1, 6144 // dim), "dim": dim,
                "rotary": 2 * rng.randint(1, dim // 2) if rng.random() < 0.3 else rng.choice([dim, dim, dim // 2]),
                "layout": rng.choice(sorted(LAYOUT)), "scaling": rng.choice(["plain", "yarn"]),
                "span": _log(rng, 64, 1 << 20)}
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
    while kv_heads * (group + 2) * dim > 7168:
        kv_heads, group = max(1, kv_heads // 2), max(1, group - 1)
    heads = {"q_heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim}
    page, kv = rng.choice([16, 32, 64, 128, 256]), rng.choice(sorted(KV))
    if op == "append":
        return {"op": op, "T": _log(rng, 1, 4096), **heads, "rotary": rng.choice([dim, dim, dim // 2]),
                "layout": rng.choice(sorted(LAYOUT)), "scaling": rng.choice(["plain", "yarn"]),
                "span": _log(rng, 4096, 1 << 20), "page": page, "kv": kv}
    batch = _log(rng, 1, 256)
    longest = _log(rng, 1, max(64, min(131072, 524288 // batch)))
    spread, window = rng.choice([1, 8, 64]), rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    while True:
        case = {"op": op, "B": batch, **heads, "page": page, "kv": kv, "min_len": max(1, longest // spread),
                "max_len": longest, "window": window}
        if work({**case, "window": 0})["bytes"] <= 5e8:
            return case
        longest //= 2


def _lengths(case):
    """The batch's lengths: spread over the logarithm between the two ends, the same for every seed."""
    low, high = case["min_len"], case["max_len"]
    ratio = high / low
    got = [int(round(low * ratio ** (((i + 1) * 0.6180339887498949) % 1.0))) for i in range(case["B"])]
    got[case["B"] // 2] = high
    return got


def _frequencies(case):
    """Radians per position of each pair, and the factor on the rotated values."""
    n, base = case["rotary"] // 2, 1e6
    f = base ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))
    if case["scaling"] == "plain":
        return f, 1.0
    # YaRN: slow pairs are stretched by `factor`, fast ones kept, a ramp between
    factor, original = 4.0, 32768.0
    where = [n * math.log(original / (turns * 2 * math.pi)) / math.log(base) for turns in (32.0, 1.0)]
    low, high = max(math.floor(where[0]), 0), min(math.ceil(where[1]), 2 * n - 1)
    ramp = ((torch.arange(n, dtype=torch.float64) - low) / max(high - low, 1e-3)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0


def _pack(fmt, t):
    """N x K trits (signs for q1) as the packed plane of a format."""
    N, K = t.shape
    if fmt == "q1":
        return ((t.view(N, K // 8, 8) > 0) * torch.tensor([1, 2, 4, 8, 16, 32, 64, 128], device=t.device)).sum(-1).to(torch.uint8)
    if fmt == "ptq1":
        d = torch.nn.functional.pad(t.view(N, K // 128, 128) + 1, (0, 2)).view(N, K // 128, 26, 5)
        return (d * torch.tensor([1, 3, 9, 27, 81], device=t.device)).sum(-1).to(torch.uint8).view(N, -1)
    return ((t.view(N, K // 4, 4) + 1) * torch.tensor([1, 4, 16, 64], device=t.device)).sum(-1).to(torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = dict(case)
    if case["op"] == "linear":
        M, N, K, fmt = case["M"], case["N"], case["K"], case["fmt"]
        u = torch.rand((N, K), generator=g, device=dev)
        t = (u > 0.69).to(torch.int8) - (u < 0.31).to(torch.int8) if fmt != "q1" else (u > 0.5).to(torch.int8) * 2 - 1
        s["packed"] = _pack(fmt, t).contiguous()
        groups = K // (64 if fmt == "pq2g64" else 128)
        s["scales"] = (0.01 + 0.04 * torch.rand((N, groups), generator=g, device=dev)).half()
        s["x"] = normal(M, K).half()
        s["b"] = normal(N).half() if case["bias"] else None
        s["r"] = (4 * normal(M, N)).half() if case["residual"] else None
        s["y"] = torch.empty((M, N), dtype=torch.float16, device=dev)
        return s
    if case["op"] != "attend":
        f, s["magnitude"] = _frequencies(case)
        s["freqs"] = f.to(dev)
        s["positions"] = torch.randint(0, case["span"], (case["T"],), generator=g, device=dev, dtype=torch.int32)
    if case["op"] == "rope":
        s["x"] = normal(case["T"], case["heads"] * case["dim"]).half()
        s["out"] = torch.empty_like(s["x"])
        return s
    H, D, page = case["kv_heads"], case["dim"], case["page"]
    kind = torch.float16 if case["kv"] == "f16" else torch.float8_e4m3fn
    s["k_scale"] = s["v_scale"] = None
    if case["kv"] == "e4m3":  # a scale per head, as a calibration run gives: the largest value seen over 448
        s["k_scale"], s["v_scale"] = ((0.008 + 0.008 * torch.rand(H, generator=g, device=dev)) for _ in range(2))
    if case["op"] == "append":
        T, pages = case["T"], (case["T"] + page - 1) // page * 5 // 4 + 1
        s["qkv"] = normal(T, (case["q_heads"] + 2 * H) * D).half()
        s["slots"] = torch.randperm(pages * page, generator=g, device=dev)[:T].contiguous()
        s["q_out"] = torch.empty((T, case["q_heads"] * D), dtype=torch.float16, device=dev)
        s["k_cache"] = torch.zeros((pages, H, page, D), device=dev).to(kind)
        s["v_cache"] = torch.zeros((pages, H, page, D), device=dev).to(kind)
        return s
    lengths = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
    need = (lengths + page - 1) // page
    width, pages = (case["max_len"] + page - 1) // page, sum((n + page - 1) // page for n in _lengths(case))
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)  # pages as an allocator hands them out
    at = torch.arange(width, device=dev)[None] + (torch.cumsum(need, 0) - need)[:, None]
    used = torch.arange(width, device=dev)[None] < need[:, None]
    s["table"] = torch.where(used, order[at.clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    s["lengths"] = lengths
    s["q"] = (2 * normal(case["B"], case["q_heads"] * D)).half()
    s["out"] = torch.empty((case["B"], case["q_heads"] * D), dtype=torch.float16, device=dev)
    s["k_cache"], s["v_cache"] = ((torch.randn((pages, H, page, D), generator=g, device=dev, dtype=torch.float16)
                                   if c is None else (normal(pages, H, page, D) / c[:, None, None]).clamp(-448, 448).to(kind))
                                  for c in (s["k_scale"], s["v_scale"]))
    return s


# ------------------------------------------------------------------ the plain forms

def _trits(fmt, packed, N, K):
    if fmt == "q1":
        return ((packed[..., None] >> torch.arange(8, device=packed.device)) & 1).view(N, K) * 2 - 1
    if fmt == "ptq1":
        p = torch.tensor([1, 3, 9, 27, 81], device=packed.device)
        return (packed.view(N, K // 128, 26, 1).int() // p % 3).view(N, K // 128, 130)[..., :128].reshape(N, K) - 1
    return ((packed[..., None] >> (2 * torch.arange(4, device=packed.device))) & 3).view(N, K).int() - 1


def _activate(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _linear(s):
    M, N, K = s["M"], s["N"], s["K"]
    h2 = torch.tensor([[1.0, 1.0], [1.0, -1.0]], device=s["x"].device)
    h = functools.reduce(torch.kron, [h2] * 7) / math.sqrt(128.0)
    xr = (s["x"].float().view(-1, 128) @ h).view(M, K)
    w = _trits(s["fmt"], s["packed"], N, K).float()
    w = (w.view(N, s["scales"].shape[1], -1) * s["scales"].float()[..., None]).view(N, K)
    y = xr @ w.t()
    if s["b"] is not None:
        y = y + s["b"].float()
    y = _activate(y, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.half()


def _rotate(x, s):
    """T x heads x dim values rotated, in 32 bits; the angles in 64."""
    R = s["rotary"]
    angle = s["positions"].double()[:, None] * s["freqs"]
    c, n = (s["magnitude"] * torch.cos(angle)).float()[:, None], (s["magnitude"] * torch.sin(angle)).float()[:, None]
    x = x.float()
    if s["layout"] == "half":
        a, b = x[..., : R // 2], x[..., R // 2: R]
        return torch.cat([a * c - b * n, b * c + a * n, x[..., R:]], -1)
    a, b = x[..., 0:R:2], x[..., 1:R:2]
    return torch.cat([torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2), x[..., R:]], -1)


def _append(s):
    T, Hq, H, D, page = s["T"], s["q_heads"], s["kv_heads"], s["dim"], s["page"]
    x = s["qkv"].view(T, Hq + 2 * H, D)
    r = _rotate(x[:, : Hq + H], s)
    s["q_out"].copy_(r[:, :Hq].half().view(T, Hq * D))
    k, v = r[:, Hq:], x[:, Hq + H:].float()
    if s["kv"] == "e4m3":
        k, v = (k / s["k_scale"][:, None]).clamp(-448, 448), (v / s["v_scale"][:, None]).clamp(-448, 448)
    p, o = s["slots"] // page, s["slots"] % page
    # (indexed writes of 8-bit floats go through their bytes)
    kind, bits = s["k_cache"].dtype, torch.uint8 if s["kv"] == "e4m3" else torch.int16
    s["k_cache"].view(bits)[p, :, o] = k.to(kind).view(bits)
    s["v_cache"].view(bits)[p, :, o] = v.to(kind).view(bits)
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _attend(s):
    B, H, D = s["B"], s["kv_heads"], s["dim"]
    G = s["q_heads"] // H
    at = s["table"].clamp(min=0).long()
    bits = torch.uint8 if s["kv"] == "e4m3" else torch.int16
    k, v = (c.view(bits)[at].view(c.dtype).float().transpose(1, 2).reshape(B, H, -1, D) for c in (s["k_cache"], s["v_cache"]))
    if s["kv"] == "e4m3":
        k, v = k * s["k_scale"][:, None, None], v * s["v_scale"][:, None, None]
    z = (s["q"].float().view(B, H, G, D) @ k.transpose(2, 3)) / math.sqrt(D)
    j, n = torch.arange(z.shape[-1], device=z.device)[None], s["lengths"][:, None]
    live = (j < n) & (j >= n - s["window"]) if s["window"] else j < n
    z = torch.where(live[:, None, None], z, -math.inf)
    e = torch.exp(z - z.amax(-1, keepdim=True))
    return ((e @ v) / e.sum(-1, keepdim=True)).half().view(B, -1)


def run(state):
    s = state
    if own:
        from ternary_weight_02_b200 import bonsai as bz
        if s["op"] == "linear":
            bz.bonsai_ternary_linear_epilogue(s["x"], s["packed"], s["scales"], s["b"], s["r"], s["y"], s["M"], s["N"],
                                              s["K"], FMT[s["fmt"]], ACT[s["act"]])
            return s["y"]
        if s["op"] == "rope":
            bz.bonsai_rope(s["x"], s["out"], s["freqs"], s["positions"], s["T"], s["heads"], s["dim"], s["rotary"],
                           LAYOUT[s["layout"]], magnitude=s["magnitude"])
            return s["out"]
        if s["op"] == "append":
            bz.bonsai_rope_append(s["qkv"], s["q_out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                  s["freqs"], s["positions"], s["slots"], s["T"], s["q_heads"], s["rotary"],
                                  LAYOUT[s["layout"]], magnitude=s["magnitude"])
            return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}
        bz.bonsai_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                  s["lengths"], s["out"], s["B"], s["q_heads"], window=s["window"])
        return s["out"]
    if s["op"] == "linear":
        return _linear(s)
    if s["op"] == "rope":
        T = s["T"]
        return _rotate(s["x"].view(T, s["heads"], s["dim"]), s).half().view(T, -1)
    return _append(s) if s["op"] == "append" else _attend(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        plane = N * K // 128 * {"ptq1": 26 + 2, "pq2": 32 + 2, "q1": 16 + 2, "pq2g64": 32 + 4}[case["fmt"]]
        return {"bytes": plane + 2 * (M * K + M * N * (2 if case["residual"] else 1) + (N if case["bias"] else 0)),
                "flops": 2 * M * N * K}
    if case["op"] == "rope":
        n = case["T"] * case["heads"] * case["dim"]
        return {"bytes": 4 * n + 4 * case["T"] + 4 * case["rotary"], "flops": 3 * n}
    wide = 1 if case["kv"] == "e4m3" else 2
    if case["op"] == "append":
        q, kv = case["T"] * case["q_heads"] * case["dim"], 2 * case["T"] * case["kv_heads"] * case["dim"]
        return {"bytes": 4 * q + (2 + wide) * kv + 12 * case["T"], "flops": 3 * q + 3 * kv // 2}
    keys = sum(min(n, case["window"] or n) for n in _lengths(case))
    return {"bytes": 2 * wide * keys * case["kv_heads"] * case["dim"] + 4 * case["B"] * case["q_heads"] * case["dim"]
            + 4 * sum((n + case["page"] - 1) // case["page"] for n in _lengths(case)),
            "flops": 4 * keys * case["q_heads"] * case["dim"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def _codebook(fmt):
    """Weights of each byte value, least significant first."""
    rows = []
    for byte in range(256):
        if fmt == "ptq1":
            digits = [byte // 3 ** i % 3 - 1 for i in range(5)]
        elif fmt == "q1":
            digits = [2 * (byte >> i & 1) - 1 for i in range(8)]
        else:
            digits = [(byte >> 2 * i & 3) - 1 for i in range(4)]
        rows.append(digits)
    return torch.tensor(rows, dtype=torch.float64)


def _exact_linear(s):
    M, N, K, fmt = s["M"], s["N"], s["K"], s["fmt"]
    dev = s["x"].device
    i = torch.arange(128, device=dev)
    parity = torch.zeros((128, 128), dtype=torch.int64, device=dev)
    for bit in range(7):
        parity ^= (i[:, None] >> bit) & (i[None] >> bit) & 1
    h = (1 - 2 * parity).double() / 128 ** 0.5
    w = _codebook(fmt).to(dev)[s["packed"].long().view(-1)].view(N, K // 128, -1)[..., :128].reshape(N, K)
    per = K // s["scales"].shape[1]
    w = w * s["scales"].double().repeat_interleave(per, 1)
    # the rotation taken to the weights: W (H x) = (W H) x, H symmetric
    w = torch.einsum("ngi,ij->ngj", w.view(N, K // 128, 128), h).reshape(N, K)
    y = torch.einsum("mk,nk->mn", s["x"].double(), w)
    if s["b"] is not None:
        y += s["b"].double()[None]
    a = s["act"]
    if a == "relu":
        y = torch.maximum(y, torch.zeros_like(y))
    elif a == "silu":
        y = y * torch.sigmoid(y)
    elif a == "gelu":
        y = y * 0.5 * torch.erfc(-y / 2 ** 0.5)
    elif a == "gelu_tanh":
        y = y * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (y + 0.044715 * y ** 3))
    return y if s["r"] is None else y + s["r"].double()


def _exact_rotated(x, s):
    """Each pair as a complex number times magnitude * e^(i angle)."""
    R = s["rotary"]
    y = x.double().clone()
    if R:
        half = s["layout"] == "half"
        a, b = (y[..., : R // 2], y[..., R // 2: R]) if half else (y[..., 0:R:2], y[..., 1:R:2])
        turn = torch.polar(torch.full_like(s["freqs"], s["magnitude"]).expand(s["T"], -1).contiguous(),
                           torch.outer(s["positions"].double(), s["freqs"]))
        z = torch.complex(a.contiguous(), b.contiguous()) * turn[:, None]
        if half:
            y[..., : R // 2], y[..., R // 2: R] = z.real, z.imag
        else:
            y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "linear":
        return _exact_linear(s)
    if s["op"] == "rope":
        return _exact_rotated(s["x"].view(s["T"], s["heads"], s["dim"]), s).view(s["T"], -1)
    H, D, page = s["kv_heads"], s["dim"], s["page"]
    if s["op"] == "append":
        T, Hq = s["T"], s["q_heads"]
        x = s["qkv"].view(T, -1, D)
        q, k, v = _exact_rotated(x[:, :Hq], s), _exact_rotated(x[:, Hq:Hq + H], s), x[:, Hq + H:].double()
        if s["kv"] == "e4m3":  # in units of the head's scale, not yet rounded to 8 bits
            k, v = ((c / f.double()[None, :, None]).clamp(-448, 448) for c, f in ((k, s["k_scale"]), (v, s["v_scale"])))
        pools = []
        for c in (k, v):
            pool = torch.zeros((s["k_cache"].shape[0] * page, H, D), dtype=torch.float64, device=c.device)
            pool[s["slots"]] = c
            pools.append(pool.view(-1, page, H, D).transpose(1, 2).contiguous())
        return {"q": q.view(T, -1), "k": pools[0], "v": pools[1]}
    out = torch.zeros((s["B"], s["q_heads"], D), dtype=torch.float64, device=s["q"].device)
    G = s["q_heads"] // H
    for b, n in enumerate(_lengths(case)):
        pages = s["table"][b, : (n + page - 1) // page].long()
        first = max(0, n - s["window"]) if s["window"] else 0
        bits = torch.uint8 if s["kv"] == "e4m3" else torch.int16
        k, v = (c.view(bits)[pages].view(c.dtype).double().permute(1, 0, 2, 3).reshape(H, -1, D)[:, first:n]
                for c in (s["k_cache"], s["v_cache"]))
        if s["kv"] == "e4m3":
            k, v = k * s["k_scale"].double()[:, None, None], v * s["v_scale"].double()[:, None, None]
        z = torch.einsum("hgd,hnd->hgn", s["q"][b].double().view(H, G, D), k) * D ** -0.5
        out[b] = torch.einsum("hgn,hnd->hgd", torch.softmax(z, -1), v).reshape(-1, D)
    return out.view(s["B"], -1)
