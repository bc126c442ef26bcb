"""The serving operators' definition in 64 bits (numpy), for the tests: the
paged 8-bit cache (a scale for 16 tokens and a head), the rotation, attention
over it, and 4-bit weights. Written from the formulas."""
import numpy as np

from oracle import E4M3, encode
from oracle.formats import decode_table

TOK = 16
VALUES = decode_table(E4M3)


def bias_of(amax, most=448.0):
    """floor(log2(most / amax)), clamped; 126 for 0."""
    if amax == 0:
        return 126
    b = int(np.floor(np.log2(most) - np.log2(amax))) + 1
    while np.ldexp(amax, b) > most:
        b -= 1
    return max(-126, min(126, b))


def need_of(x):
    """What new values ask of their block's bias."""
    fin = np.abs(x[np.isfinite(x)])
    b = bias_of(float(fin.max()) if fin.size else 0.0)
    return min(b, 0) if np.isinf(x).any() else b


def rotate(x, pos, freqs, inter):
    """x [tokens, heads, d] at positions pos; freqs (float32 values) or None."""
    x = np.array(x, dtype=np.float64)
    if freqs is None or len(freqs) == 0:
        return x
    r = 2 * len(freqs)
    t = np.asarray(pos, dtype=np.float64)[:, None, None] * np.asarray(freqs, dtype=np.float64)
    c, s = np.cos(t), np.sin(t)
    i, j = (np.arange(0, r, 2), np.arange(1, r, 2)) if inter else (np.arange(r // 2), np.arange(r // 2, r))
    a, b = x[..., i].copy(), x[..., j].copy()
    x[..., i], x[..., j] = a * c - b * s, b * c + a * s
    return x


class Model:
    """A cache's state: codes [pages, slots, heads, d] and biases [pages, blocks, heads], for keys and values."""

    def __init__(self, pages, page, heads, d):
        self.page, self.pages = page, pages
        self.codes = np.zeros((2, pages, page, heads, d), dtype=np.uint8)
        self.bias = np.full((2, pages, page // TOK, heads), 127, dtype=np.int64)    # nothing stored: scale byte 0

    def place(self, table, pos):
        """(page, slot) of a position, or None."""
        if pos < 0 or pos // self.page >= len(table):
            return None
        p = int(table[pos // self.page])
        return (p, pos % self.page) if 0 <= p < self.pages else None

    def append(self, k, v, tables, lengths, starts=None, freqs=None, inter=False):
        """k, v [tokens, heads, d] (64 bits)."""
        starts = np.arange(len(lengths) + 1) if starts is None else starts
        for i, length in enumerate(lengths):
            r0, r1 = int(starts[i]), int(starts[i + 1])
            p0 = max(0, int(length)) - (r1 - r0)
            pos = np.arange(p0, p0 + r1 - r0)
            both = (rotate(k[r0:r1], pos, freqs, inter), np.asarray(v[r0:r1], dtype=np.float64))
            for b in sorted(set(int(p) // TOK for p in pos if p >= 0)):
                at = self.place(tables[i], b * TOK)
                if at is None:
                    continue
                rows = [j for j, p in enumerate(pos) if p // TOK == b]
                first, blk, page = int(pos[rows[0]]) % TOK, at[1] // TOK, at[0]
                base = at[1]
                for w in range(2):
                    x = both[w][rows]
                    for h in range(x.shape[1]):
                        bias = need_of(x[:, h])
                        was = int(self.bias[w, page, blk, h])
                        if first:
                            bias = min(bias, was)
                            if bias < was:
                                old = self.codes[w, page, base:base + first, h]
                                old[:] = encode(VALUES[old] * (0.0 if was == 127 else 2.0 ** (bias - was)), E4M3)
                        most = 240.0 if bias == -120 else 448.0                       # finite in bf16
                        with np.errstate(over="ignore"):
                            y = np.clip(x[:, h] * 2.0 ** bias, -most, most)
                        self.codes[w, page, base + first:base + first + len(rows), h] = encode(y, E4M3)
                        self.bias[w, page, blk, h] = bias

    def values(self, w, table, pos):
        """[positions, heads, d], zeros where there is no page; and which positions are there."""
        out = np.zeros((len(pos), *self.codes.shape[3:]))
        there = np.zeros(len(pos), dtype=bool)
        for n, p in enumerate(pos):
            at = self.place(table, int(p))
            if at:
                there[n] = True
                b = self.bias[w, at[0], at[1] // TOK]
                out[n] = VALUES[self.codes[w, at[0], at[1]]] * np.where(b == 127, 0.0, 2.0 ** -b.astype(np.float64))[:, None]
        return out, there

    def read(self, tables, lengths, starts=None):
        starts = np.arange(len(lengths) + 1) if starts is None else starts
        out = [[], []]
        for i, length in enumerate(lengths):
            n = int(starts[i + 1] - starts[i])
            p0 = max(0, int(length)) - n
            for w in range(2):
                out[w].append(self.values(w, tables[i], np.arange(p0, p0 + n))[0])
        return np.concatenate(out[0]), np.concatenate(out[1])


def attend(q, model, tables, lengths, starts=None, scale=None, softcap=0.0, window=0):
    """(out, lse, slack) of q [tokens, hq, d]: slack is sum p |v| and, in [..., -1], the largest sum of |q k| scale of a
    seen score: what roundings of the weights and of the scores scale with."""
    t, hq, d = q.shape
    g = hq // model.codes.shape[3]
    scale = d ** -0.5 if scale is None else scale
    starts = np.arange(len(lengths) + 1) if starts is None else starts
    out, lse = np.zeros((t, hq, d)), np.full((t, hq), -np.inf)
    mass, size = np.zeros((t, hq, d)), np.zeros((t, hq))
    for i, length in enumerate(lengths):
        r0, r1 = int(starts[i]), int(starts[i + 1])
        length = max(0, int(length))
        k, there = model.values(0, tables[i], np.arange(length))
        v, _ = model.values(1, tables[i], np.arange(length))
        for r in range(r0, r1):
            p = length - (r1 - r0) + r - r0
            j = np.arange(length)
            seen = there & (j <= p) & ((j > p - window) if window else True)
            if not seen.any():
                continue
            for h in range(hq):
                with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
                    s = k[seen, h // g] @ q[r, h] * scale
                    size[r, h] = np.max(np.abs(k[seen, h // g]) @ np.abs(q[r, h])) * abs(scale)
                    if softcap:
                        s = softcap * np.tanh(s / softcap)
                    e = np.exp(s - s.max())
                    w = e / e.sum()
                    out[r, h] = w @ v[seen, h // g]
                    mass[r, h] = w @ np.abs(v[seen, h // g])
                    lse[r, h] = s.max() + np.log(e.sum())
    return out, lse, mass, size


# Roundings between scores and outputs, relative to sum p |v|: each weight to bf16 (2^-8); a score's product of d terms in
# 32 bits, at most d + 2 additions and products of 2^-24 each; scaling, softcap and base-2 logarithm (8 roundings of the
# score, and tanh within 2^-20), 2^-20 of exp2. A score's error e changes weights and their sum by e each.
def tolerance(out, mass, size, d):
    score = size * ((d + 10) * 2.0 ** -24 + 2.0 ** -20)
    return 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -18 + 2 * score)[..., None] * mass * 1.01 + 2.0 ** -133


GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


MIDDLES = (GRID[1:] + GRID[:-1]) / 2


def fp4_codes(w):
    """codes (0 .. 15) and biases of w [K, N], groups of 32 along K; a group with a NaN has bias nan."""
    w = np.asarray(w, dtype=np.float64)
    K, N = w.shape
    g = -(-K // 32)
    p = np.zeros((g * 32, N))
    p[:K] = w
    p = p.reshape(g, 32, N)
    with np.errstate(invalid="ignore"):
        a = np.abs(p).max(1)
    ok = np.isfinite(a) & (a > 0)
    m, e = np.frexp(np.where(ok, a, 1.0))
    b = np.where(ok, np.clip(3 - e - (m > 0.75), -126, 126), 0)           # 6 = 0.75 2^3
    assert ((a * 2.0 ** b <= 6) | ~ok | (b == -126)).all() and ((a * 2.0 ** (b + 1) > 6) | ~ok | (b == 126)).all()
    y = np.minimum(np.abs(p) * 2.0 ** b[:, None], 6.0)
    codes = np.zeros(p.shape, dtype=np.uint8)
    for i, mid in enumerate(MIDDLES):
        codes += (y >= mid) if i % 2 else (y > mid)                       # a middle goes to the even code
    return codes | (np.signbit(p).astype(np.uint8) << 3), np.where(np.isnan(a), np.nan, b)


def fp4_held(w):
    """The values of w's 4-bit form."""
    codes, bias = fp4_codes(w)
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0) * 2.0 ** -bias[:, None, :]
    return v.reshape(-1, w.shape[1])[:w.shape[0]]
