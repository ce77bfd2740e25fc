"""Plain numpy oracles of the attention half of a decode step, in 64 bits:
head norms and rotation, the 4-bit cache's quantizer and layout, and the
attention over it.  They share no code with the HIP path.  Test
infrastructure only."""
import numpy as np

F16_STEP = 2.0 ** -25  # half of binary16's least step


def norm_rope(x, w, eps, positions, inv_freq, interleaved):
    """x [T, H, D] float64 -> (y, bound): the result in 64 bits and, per
    element, the sum of the magnitudes that its last step adds up."""
    y = np.array(x, np.float64)
    if w is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    rot = 2 * len(inv_freq)
    a = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float32).astype(np.float64)
    cos, sin = np.cos(a)[:, None, :], np.sin(a)[:, None, :]
    mag = np.abs(y)
    lo, hi = (np.s_[..., 0:rot:2], np.s_[..., 1:rot:2]) if interleaved else (np.s_[..., :rot // 2], np.s_[..., rot // 2:rot])
    u, v = y[lo].copy(), y[hi].copy()
    y[lo], y[hi] = u * cos - v * sin, v * cos + u * sin
    mag[lo] = mag[hi] = np.abs(u) + np.abs(v)
    return y, mag


def quantize(x):
    """Codes, scale and middle of every head (the last axis): each step fp32."""
    x = np.asarray(x, np.float32)
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    z = ((hi + lo) * np.float32(0.5)).astype(np.float16)
    s = ((hi - lo) / np.float32(15)).astype(np.float16)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.rint((x - z.astype(np.float32)) / s.astype(np.float32) + np.float32(7.5))
    c = np.where(s == 0, 0, np.clip(np.nan_to_num(c), 0, 15)).astype(np.uint8)
    return c, s[..., 0], z[..., 0]


def held(c, s, z):
    """The value that a code stands for, in 64 bits."""
    s, z = s.astype(np.float64)[..., None], z.astype(np.float64)[..., None]
    return np.where(s == 0, z + 0 * c, z + s * (c.astype(np.float64) - 7.5))


class Cache:
    """A paged cache as bytes, [pages, Hk, P*(D+8)], with its layout written
    out entry by entry."""

    def __init__(self, pages, Hk, P, D, fill=0):
        self.P, self.D, self.Hk, self.pages = P, D, Hk, pages
        self.bytes = np.full((pages, Hk, P * (D + 8)), fill, np.uint8)

    def _value_byte(self, t, d):
        unit = ((t // 32) * 4 + (t % 32) // 8) * (self.D // 4) + d // 4
        return self.P * self.D // 2 + (unit * 8 + t % 8) * 2 + (d % 4) // 2

    def put(self, slot, head, value, c, s, z):
        b, t = self.bytes[slot // self.P, head], slot % self.P
        for d in range(self.D):
            at = self._value_byte(t, d) if value else t * (self.D // 2) + d // 2
            keep = 0x0f if d % 2 else 0xf0
            b[at] = (b[at] & keep) | (int(c[d]) << (4 * (d % 2)))
        at = self.P * (self.D + 4 * bool(value)) + 4 * t
        b[at:at + 2] = np.frombuffer(np.float16(s).tobytes(), np.uint8)
        b[at + 2:at + 4] = np.frombuffer(np.float16(z).tobytes(), np.uint8)

    def get(self, slot, head, value):
        b, t = self.bytes[slot // self.P, head], slot % self.P
        d = np.arange(self.D)
        at = self._value_byte(t, d) if value else t * (self.D // 2) + d // 2
        c = (b[at] >> (4 * (d % 2))) & 15
        at = self.P * (self.D + 4 * bool(value)) + 4 * t
        s, z = np.frombuffer(b[at:at + 4].tobytes(), np.float16)
        return c, s, z

    def store(self, k, v, slots):
        for t, slot in enumerate(slots):
            if 0 <= slot < self.pages * self.P:
                for h in range(self.Hk):
                    for value, x in ((0, k), (1, v)):
                        c, s, z = quantize(x[t, h])
                        self.put(int(slot), h, value, c, s, z)

    def tokens(self, slots, head):
        """Codes, scales and middles of keys and of values, slot by slot."""
        out = []
        for value in (0, 1):
            got = [self.get(int(s), head, value) for s in slots]
            out.append(tuple(np.array([g[i] for g in got]).reshape((len(got), self.D) if i == 0 else (len(got),))
                             for i in range(3)))
        return out


def attention(q, cache, table, ctx_len, q_start, scale, window, eps, kept=None):
    """(out, lse, out tolerance, lse tolerance) of q [T, Hq, D] (float64
    values) for an output type of half step eps/2.  Tolerances: half a step of
    the output; 16 fp32 roundings of the magnitudes in a score; fp32 sums of n
    terms over 32 accumulators with their fixed parts (n/32 + 64); and for the
    p*s that go to the matrix cores in binary16:
      kept given (2^-22 with the rounding's remainder, 2^-11 without): that of
      every |p s (c - 7.5)|, and half a binary16 step for each in units where
      the row's largest p*s is at least 2^4, or the largest p 2^30;
      else 2^-11 of every |p s (c - 7.5)| and half a step in units where the
      largest s, whatever its p, is 8 (which is wide where the scales of a row
      differ by far)."""
    T, Hq, D = q.shape
    G = Hq // cache.Hk
    out, lse = np.full(q.shape, np.nan), np.full((T, Hq), np.nan)
    tol, ltol = np.zeros(q.shape), np.zeros((T, Hq))
    for b in range(len(ctx_len)):
        t0, n, c = q_start[b], q_start[b + 1] - q_start[b], int(ctx_len[b])
        j = np.arange(c)
        page = table[b][j // cache.P] if c else j
        good = (page >= 0) & (page < cache.pages)
        slots = np.where(good, page * cache.P + j % cache.P, 0)
        for h in range(cache.Hk):
            (kc, ks, kz), (vc, vs, vz) = cache.tokens(slots, h)
            with np.errstate(invalid="ignore"):
                k, v = held(kc, ks, kz), held(vc, vs, vz)
                vs64 = vs.astype(np.float64)[:, None]
                centred = np.abs(vs64 * (vc - 7.5))
                kmag = 7.5 * np.abs(ks.astype(np.float64)) + np.abs(kz.astype(np.float64))
                vmag = 15 * np.abs(vs64[:, 0]) + np.abs(vz.astype(np.float64))
            for i in range(n):
                p0 = c - n + i
                see = good & (j <= p0)
                if window:
                    see &= j > p0 - window
                for g in range(G):
                    hq = h * G + g
                    if not see.any():
                        out[t0 + i, hq], lse[t0 + i, hq] = 0, -np.inf
                        continue
                    x = k[see] @ q[t0 + i, hq] * scale
                    top = x.max()
                    p = np.exp(x - top)
                    total = p.sum()
                    p /= total
                    o = p @ v[see]
                    out[t0 + i, hq], lse[t0 + i, hq] = o, top + np.log(total)
                    m = see.sum()
                    score = 16 * 2.0 ** -24 * (kmag[see].max() * np.abs(q[t0 + i, hq]).sum() * abs(scale) + abs(top))
                    sums = (m / 32 + 64) * 2.0 ** -24
                    if kept is None:
                        held16 = 2.0 ** -11 * (p @ centred[see]) + m / total * F16_STEP * 7.5 * vs64[see].max() / 8
                    else:
                        held16 = kept * (p @ centred[see]) + m * F16_STEP * 7.5 * max(np.max(p * vs64[see][:, 0]) / 2 ** 4,
                                                                                     p.max() * 2.0 ** -30)
                    tol[t0 + i, hq] = (eps / 2 * np.abs(o) + F16_STEP + held16
                                       + 2 * score * (p @ np.abs(v[see]) + np.abs(o)) + sums * (p @ vmag[see]))
                    ltol[t0 + i, hq] = 2 * score + sums + 2.0 ** -22 * abs(lse[t0 + i, hq])
    return out, lse, tol, ltol
