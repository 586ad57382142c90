"""Plain float64 forms of the decode layer's operators around the ternary products, and the
error bounds their kernels are held to.  Numpy only; nothing here calls the library."""
import math

import numpy as np

H16 = 2.0 ** -11        # half a step of FP16, relative
TINY16 = 2.0 ** -25     # half a step below FP16's normal range, absolute


def activate(z, act):
    z = np.asarray(z, dtype=np.float64)
    with np.errstate(over="ignore"):
        if act == 1:
            return np.where(z < 0, 0.0, z)
        if act == 2:
            return z / (1.0 + np.exp(-z))
        if act == 3:
            return z * 0.5 * np.vectorize(math.erfc)(-z / math.sqrt(2.0)) if z.size else z
        if act == 4:
            return z * 0.5 * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def frequencies(R, base, scaling="plain", factor=1.0, original=0.0, low=1.0, high=32.0):
    """Frequencies (radians per position) and magnitude, one pair at a time."""
    out = []
    if scaling == "ntk" and R > 2:
        base = base * factor ** (R / (R - 2))
    for i in range(R // 2):
        f = base ** (-2.0 * i / R)
        turns = original * f / (2 * math.pi)
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            # pair index at which f makes `t` turns over the original context
            at = lambda t: R / 2 * math.log(original / (2 * math.pi * t)) / math.log(base)  # noqa: E731
            a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), R - 1)
            r = min(max((i - a) / max(b - a, 1e-3), 0.0), 1.0)
            f = f * (1 - r) + f / factor * r
        elif scaling == "bands":
            if turns < low:
                f = f / factor
            elif turns <= high:
                s = (turns - low) / (high - low)
                f = (1 - s) * f / factor + s * f
        out.append(f)
    return np.array(out, dtype=np.float64), (1 + 0.1 * math.log(factor)) if scaling == "yarn" else 1.0


def rope(x, positions, freqs, R, layout, magnitude):
    """(T, H, D) float64 rotated, and the FP32 kernel's error bound before any rounding: the
    sine and cosine are off by 2^-22 at most (argument rounded to FP32 within half a turn,
    two units in the last place of the functions), each product and the sum by 2^-24."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    slack = np.zeros_like(x)
    for i in range(R // 2):
        a, b = (i, i + R // 2) if layout == 0 else (2 * i, 2 * i + 1)
        # the angle in extended precision, so that this reference is not the one that is off
        ang = np.asarray(positions, dtype=np.longdouble) * np.longdouble(freqs[i])
        c, s = np.asarray(np.cos(ang), np.float64)[:, None], np.asarray(np.sin(ang), np.float64)[:, None]
        y[..., a] = magnitude * (x[..., a] * c - x[..., b] * s)
        y[..., b] = magnitude * (x[..., b] * c + x[..., a] * s)
        slack[..., a] = slack[..., b] = 2.0 ** -20 * magnitude * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, slack


def f16_bound(ref, slack):
    return H16 * np.abs(ref) + TINY16 + slack * (1 + H16)


def e4m3_values(codes):
    """Values of e4m3 bytes, from the format's definition."""
    codes = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    sign = np.where(codes & 0x80, -1.0, 1.0)
    e, m = (codes >> 3) & 15, codes & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where((codes & 0x7f) == 0x7f, np.nan, sign * v)


def e4m3_bound(units, slack_units):
    """Bound on an E4M3 entry against its value in units of the scale: half a step, 2^-4
    relative or 2^-10 below the normal range (2^-6), and the FP32 error and division."""
    return 2.0 ** -4 * np.abs(units) + 2.0 ** -10 + slack_units + 2.0 ** -22 * np.abs(units)


def attention(q, k, v, lengths, window, scale):
    """One token per sequence: q (B, Hq, D); k, v lists of (len_b, Hkv, D) float64 arrays.

    Returns out, lse and bounds on both for a kernel that keeps scores and sums in FP32 and
    rounds each probability to FP16.  With S = sum |q k| scale, a score is off by at most
    d = (D + 4) 2^-24 S (D-term FP32 sum of exact products, scale and exponent base); each
    probability is then off by 2 d + 2^-20 relative (exponential and rescalings) and by its
    rounding, 2^-11 relative or 2^-25 absolute below FP16's normal range; the joined sums
    add n-independent 2^-20.  The output is rounded once more."""
    B, Hq, D = q.shape
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    tol, lse_tol = np.full((B, Hq, D), TINY16), np.zeros((B, Hq))
    for b in range(B):
        n = lengths[b]
        first = max(0, n - window) if window else 0
        if n == 0:
            continue
        kb, vb = k[b][first:n], v[b][first:n]
        G = Hq // kb.shape[1]
        for h in range(Hq):
            kk, vv, qq = kb[:, h // G], vb[:, h // G], q[b, h]
            z = kk @ qq * scale
            top = z.max()
            p = np.exp(z - top)
            l = p.sum()
            out[b, h] = p @ vv / l
            lse[b, h] = top + math.log(l)
            d = (D + 4) * 2.0 ** -24 * (np.abs(kk) @ np.abs(qq)) * abs(scale)
            r = 2 * d + 2.0 ** -20
            rel = H16 + r
            num = (p * rel) @ np.abs(vv) + 2.0 ** -25 * np.abs(vv).sum(0)
            den = (p * r).sum() / l
            tol[b, h] = num / l + den * np.abs(out[b, h]) + H16 * np.abs(out[b, h]) + TINY16
            lse_tol[b, h] = d.max() + den + 2.0 ** -20 + 2.0 ** -22 * abs(lse[b, h])
    return out, lse, tol, lse_tol


class Pool:
    """A paged cache on the host: float64 entries behind their stored bits, everything outside the
    sequences NaN."""

    def __init__(self, rng, lengths, Hkv, D, page, kv, spare=3, window=0):
        self.lengths, self.Hkv, self.D, self.page, self.kv = list(lengths), Hkv, D, page, kv
        need = [-(-n // page) for n in self.lengths]
        self.pages = sum(need) + spare
        self.width = max(need + [1]) + 1
        order = rng.permutation(self.pages)
        self.table = np.full((len(need), self.width), -1, dtype=np.int32)
        bits = np.uint8 if kv else np.uint16
        nan = 0x7f if kv else 0x7e00
        shape = (self.pages, Hkv, page, D)
        self.kbits, self.vbits = np.full(shape, nan, bits), np.full(shape, nan, bits)
        self.k_scale = rng.uniform(0.01, 0.05, Hkv).astype(np.float32) if kv else None
        self.v_scale = rng.uniform(0.01, 0.05, Hkv).astype(np.float32) if kv else None
        self.k, self.v = [], []
        at = 0
        for b, n in enumerate(self.lengths):
            self.table[b, : need[b]] = order[at: at + need[b]]
            at += need[b]
            first = max(0, n - window) if window else 0
            vals = []
            for pool, sc in ((self.kbits, self.k_scale), (self.vbits, self.v_scale)):
                if kv:
                    codes = rng.integers(0, 256, (n, Hkv, D)).astype(np.uint8)
                    codes = np.where((codes & 0x7f) >= 0x70, codes & 0x8f | 0x28, codes)  # |code| < 128: real data's range
                    full = e4m3_values(codes) * sc[None, :, None].astype(np.float64)
                    stored = codes
                else:
                    full = rng.normal(0, 1, (n, Hkv, D)).astype(np.float16)
                    stored = full.view(np.uint16)
                    full = full.astype(np.float64)
                for j in range(first, n):
                    pool[self.table[b, j // page], :, j % page] = stored[j]
                vals.append(full)
            # pages wholly before a window are free to be reused: the table may hold anything there
            self.table[b, : first // page] = -7
            self.k.append(vals[0])
            self.v.append(vals[1])

    def device(self):
        import torch
        kind = torch.float8_e4m3fn if self.kv else torch.float16
        view = np.uint8 if self.kv else np.int16
        pools = [torch.from_numpy(p.view(view)).cuda().view(kind) for p in (self.kbits, self.vbits)]
        scales = [None if s is None else torch.from_numpy(s).cuda() for s in (self.k_scale, self.v_scale)]
        return (*pools, *scales, torch.from_numpy(self.table).cuda(),
                torch.tensor(self.lengths, dtype=torch.int32, device="cuda"))
