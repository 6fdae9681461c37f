"""The microscaled cache, attention over it and the verification of drafts, from their definitions in
64 bits with numpy: what the GPU tests compare with. Slow and plain; shares nothing with the library."""
import numpy as np

MXFP8, MXFP4 = 0, 1


def magnitudes(fmt):
    """The element type's non-negative numbers, by code."""
    if fmt == MXFP4:
        return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6.0])
    return np.array([k * 2.0 ** -9 if k < 8 else (1 + k % 8 / 8) * 2.0 ** (k // 8 - 7) for k in range(127)])


def encode(x, fmt):
    """(codes uint8, exponent bytes uint8) of x[..., dim]: blocks of 32 channels."""
    x = np.asarray(x, np.float64)
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    mag, largest = magnitudes(fmt), 448.0 if fmt == MXFP8 else 6.0
    finite = np.isfinite(blocks).all(-1) & (np.abs(np.nan_to_num(blocks)).max(-1) < 2.0 ** 127)
    safe = np.where(finite[..., None], blocks, 0.0)
    top = np.abs(safe).max(-1)
    b = np.full(top.shape, 16)
    for e in range(16, 254):  # the smallest that holds the largest magnitude
        b = np.where(top > largest * 2.0 ** (e - 127), e + 1, b)
    y = np.abs(safe) * np.exp2(127.0 - b)[..., None]
    lo = np.searchsorted(mag, y, side="right") - 1  # mag[lo] <= y
    hi = np.minimum(lo + 1, len(mag) - 1)
    dl, dh = y - mag[lo], mag[hi] - y
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)) | (hi == lo), lo, hi)
    code = code + np.signbit(safe) * (128 if fmt == MXFP8 else 8)
    code = np.where(finite[..., None], code, 0)
    b = np.where(finite, b, 255)
    return code.reshape(x.shape).astype(np.uint8), b.astype(np.uint8)


def decode(code, b, fmt):
    mag = magnitudes(fmt)
    table = np.concatenate([mag, [np.nan] * (fmt == MXFP8), -mag, [np.nan] * (fmt == MXFP8)])
    b = np.repeat(b.astype(np.int64), 32, axis=-1)
    return np.where(b == 255, np.nan, table[code] * np.exp2(b - 127.0))


def record_bytes(fmt, dim):
    return (66 if fmt == MXFP8 else 34) * dim


def places(fmt, dim):
    """For token t of a record and a channel: where K's and V's code is (in codes) and where their
    exponent bytes are (in bytes)."""
    t, ch = np.arange(32)[:, None], np.arange(dim)[None]
    p, r, n = ch // 64, ch % 64, dim // 64
    a, i, h = t // 16, t % 16, r // 32
    g, tt = i // 4, i % 4
    if fmt == MXFP8:
        k = (((p * 2 + a) * 4 + r // 16) * 16 + i) * 16 + r % 16
        v = ((((p * 2 + a) * 4 + g) * 16 + r // 4) * 4 + tt) * 4 + r % 4
    else:
        k = (((p * 4 + r // 16) * 16 + i) * 2 + a) * 16 + r % 16
        v = ((((p * 4 + g) * 16 + r // 4) * 2 + a) * 4 + tt) * 4 + r % 4
    codes = 64 * dim if fmt == MXFP8 else 32 * dim
    ek = codes + ((h * 16 + i) * n + p) * 2 + a
    ev = codes + dim + (((h * 4 + g) * n + p) * 2 + a) * 4 + tt
    return k, v + 32 * dim, ek, ev


class Cache:
    """A cache's bytes on the host."""

    def __init__(self, fmt, heads, dim, page, pages, fill=0):
        self.fmt, self.heads, self.dim, self.page, self.pages = fmt, heads, dim, page, pages
        self.data = np.full(pages * heads * (page // 32) * record_bytes(fmt, dim), fill, np.uint8)
        self.at = places(fmt, dim)

    def _base(self, slot, h):
        tiles = self.page // 32
        rec = (slot // self.page * self.heads + h) * tiles + slot % self.page // 32
        return rec * record_bytes(self.fmt, self.dim)

    def write(self, k, v, slots):
        """k, v float64 [T][heads][dim]; slots outside the cache write nothing."""
        for x, code_at, exp_at in ((k, self.at[0], self.at[2]), (v, self.at[1], self.at[3])):
            code, b = encode(x, self.fmt)
            for t, slot in enumerate(slots):
                if not 0 <= slot < self.pages * self.page:
                    continue
                for h in range(self.heads):
                    base, at = self._base(slot, h), code_at[slot % 32]
                    if self.fmt == MXFP8:
                        self.data[base + at] = code[t, h]
                    else:
                        lo, hi = code[t, h, 0::2], code[t, h, 1::2]
                        self.data[base + at[0::2] // 2] = lo | (hi << 4)
                    self.data[base + exp_at[slot % 32][::32]] = b[t, h]

    def read(self, slots):
        """float64 K and V [T][heads][dim]; zeros for a slot outside the cache."""
        out = []
        for code_at, exp_at in ((self.at[0], self.at[2]), (self.at[1], self.at[3])):
            x = np.zeros((len(slots), self.heads, self.dim))
            for t, slot in enumerate(slots):
                if not 0 <= slot < self.pages * self.page:
                    continue
                for h in range(self.heads):
                    base, at = self._base(slot, h), code_at[slot % 32]
                    if self.fmt == MXFP8:
                        code = self.data[base + at]
                    else:
                        code = (self.data[base + at // 2] >> (4 * (at % 2))) & 15
                    x[t, h] = decode(code, self.data[base + exp_at[slot % 32][::32]], self.fmt)
            out.append(x)
        return out


def slots_of(table, n, page):
    return [int(table[t // page]) * page + t % page for t in range(n)]


def attend(cache, q, table, lens, prefix_table, prefix_len, scale, q_lens=None):
    """out, lse, and a bound's ingredients per row: sum w|v| / sum w (as out), the largest
    scale * sum |q k_j|, the number of tokens seen."""
    B, Q, Hq, D = q.shape
    G = Hq // cache.heads
    out, mix = np.zeros(q.shape), np.zeros(q.shape)
    lse, size = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    count = np.zeros((B, Q), np.int64)
    pk, pv = cache.read(slots_of(prefix_table, prefix_len, cache.page))
    for b in range(B):
        n = int(lens[b])
        nq = Q if q_lens is None else int(q_lens[b])
        ok, ov = cache.read(slots_of(table[b], n, cache.page))
        for i in range(nq):
            own = max(0, min(n, n - nq + i + 1))
            k, v = np.concatenate([pk, ok[:own]]), np.concatenate([pv, ov[:own]])
            count[b, i] = len(k)
            if len(k) == 0:
                continue
            for hq in range(Hq):
                h = hq // G
                s = scale * (k[:, h] @ q[b, i, hq])
                m = s.max()
                w = np.exp(s - m)
                out[b, i, hq] = w @ v[:, h] / w.sum()
                mix[b, i, hq] = w @ np.abs(v[:, h]) / w.sum()
                lse[b, i, hq] = m + np.log(w.sum())
                size[b, i, hq] = abs(scale) * (np.abs(k[:, h]) @ np.abs(q[b, i, hq])).max()
    return out, lse, mix, size, count


def verify(p, q, draft, u_accept, u_sample, n_draft=None):
    """tokens, accepted; p [B][K + 1][V], q [B][K][V] or None, exact sums in 64 bits in token order."""
    B, K = draft.shape
    V = p.shape[2]
    tokens, accepted = np.full((B, K + 1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        n = K if n_draft is None else int(n_draft[b])
        a = 0
        while a < n:
            x = int(draft[b, a])
            if not 0 <= x < V:
                break
            qx = 1.0 if q is None else float(q[b, a, x])
            if not float(u_accept[b, a]) * qx < float(p[b, a, x]):
                break
            tokens[b, a] = x
            a += 1
        target = p[b, a].astype(np.float64)
        left = None
        if a < n:
            less = np.zeros(V)
            if q is not None:
                less = q[b, a].astype(np.float64)
            elif 0 <= int(draft[b, a]) < V:
                less[int(draft[b, a])] = np.inf
            with np.errstate(invalid="ignore"):
                left = np.where(target > less, target - less, 0.0)
        if left is None or not left.sum() > 0:
            left = np.where(target > 0, target, 0.0)
        run = np.cumsum(left)
        if run[-1] > 0:
            over = np.nonzero((run > float(u_sample[b]) * run[-1]) & (left > 0))[0]
            tokens[b, a] = over[0] if len(over) else np.nonzero(left)[0][-1]
        accepted[b] = a
    return tokens, accepted
