"""Plain 64-bit model of the 4-bit key/value cache and its attention, for the tests.  It knows
the record layout from its description only: every value is looked up at its own byte and bit."""
import numpy as np

F32, F64 = np.float32, np.float64


class Layout:
    def __init__(self, D, Hk, P, g, zp):
        self.D, self.Hk, self.P, self.g, self.zp = D, Hk, P, g, zp
        self.record = P * D + 8 * P * (D // g)

    def k_at(self, p, ch):
        j, c = divmod(ch, self.g)
        q, c = divmod(c, self.g // 4)
        u, n = divmod(c, 8)
        return p * self.D // 2 + q * (self.D // 8) + j * (self.g // 8) + 4 * u + n // 2, 4 * (n % 2)

    def v_at(self, p, ch):
        n, r = divmod(ch, 16)
        h, c = divmod(n, 4)
        word = (p // 8) * self.D + h * 64 + r * 4 + (p % 8) // 2
        return self.P * self.D // 2 + 4 * word + 2 * (p % 2) + c // 2, 4 * (c % 2)

    def par_at(self, side, j, p):
        return self.P * self.D + 4 * self.P * (side * (self.D // self.g) + j) + 4 * p

    def tables(self):
        """Byte offsets and shifts [2][P][D], parameter offsets [2][P][D]."""
        if not hasattr(self, "_t"):
            at = np.zeros((2, self.P, self.D), np.int64)
            sh = np.zeros_like(at)
            par = np.zeros_like(at)
            for p in range(self.P):
                for ch in range(self.D):
                    at[0, p, ch], sh[0, p, ch] = self.k_at(p, ch)
                    at[1, p, ch], sh[1, p, ch] = self.v_at(p, ch)
                    for s in range(2):
                        par[s, p, ch] = self.par_at(s, ch // self.g, p)
            self._t = at, sh, par
        return self._t

    def decode(self, rec):
        """codes, steps, zeros (64-bit [2][P][D]) of one record (uint8 [record])."""
        at, sh, par = self.tables()
        code = (rec[at] >> sh) & 15
        h = rec.astype(np.uint16)

        def half(o):
            return (h[par + o] | (h[par + o + 1] << 8)).astype(np.uint16).view(np.float16).astype(F64)
        return code.astype(F64), half(0), half(2)

    def quantise(self, x):
        """codes, fp16 step, fp16 zero of fp32 rows [..., D] (numpy fp32 operations)."""
        v = x.astype(F32).reshape(x.shape[:-1] + (self.D // self.g, self.g))
        bad = ~np.all(np.isfinite(v), axis=-1)
        v = np.where(bad[..., None], F32(0), v)
        if self.zp:
            hi, lo = np.maximum(v.max(-1), F32(0)), np.minimum(v.min(-1), F32(0))
            with np.errstate(over="ignore"):
                st = ((hi - lo).astype(F32) / F32(15)).astype(F32)
            bad |= ~np.isfinite(st)                             # the range overflows
            v, lo, st = np.where(bad[..., None], F32(0), v), np.where(bad, F32(0), lo), np.where(bad, F32(1), st)
            st = np.where(st == 0, F32(1), st)
            z = np.clip(np.rint((-lo / st).astype(F32)), 0, 15) + F32(0)  # an integer: no -0
            c = np.clip(np.rint((v / st[..., None]).astype(F32)) + z[..., None], 0, 15)
        else:
            st = (np.abs(v).max(-1) / F32(7)).astype(F32)
            st = np.where(st == 0, F32(1), st)
            z = np.full_like(st, 8)
            c = np.clip(np.rint((v / st[..., None]).astype(F32)), -7, 7) + 8
        c = np.where(bad[..., None], 0, c).reshape(x.shape)
        with np.errstate(over="ignore"):
            s16 = np.where(bad, np.float16(np.nan), st.astype(np.float16)).astype(np.float16)
        return c.astype(np.uint8), s16, np.where(bad, 0, z).astype(np.float16)

    def write(self, rec, p, side, row):
        """Store one row (fp32 [D]) as token p of a record, in place."""
        c, s, z = self.quantise(row)
        at, sh, _ = self.tables()
        for ch in range(self.D):
            b, k = at[side, p, ch], int(sh[side, p, ch])
            rec[b] = (int(rec[b]) & (0xF0 if k == 0 else 0x0F)) | (int(c[ch]) << k)
        for j in range(self.D // self.g):
            o = self.par_at(side, j, p)
            rec[o:o + 4] = np.frombuffer(np.array([s[j], z[j]], np.float16).tobytes(), np.uint8)


def attention(lay, q, cache, table, lens, starts, scale, window):
    """64-bit out, lse and, for the tests' bounds, per row: sum p |v|, sum p step (c + z), the
    largest score error factor, number of keys.  cache uint8 [pages][Hk][record] (numpy)."""
    T, H, D = q.shape
    grp = H // lay.Hk
    out = np.zeros((T, H, D))
    lse = np.full((T, H), -np.inf)
    absv, cz = np.zeros((T, H, D)), np.zeros((T, H, D))
    dmax, keys, smax = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    memo = {}

    def rec(page, kh):
        if (page, kh) not in memo:
            memo[page, kh] = lay.decode(cache[page, kh])
        return memo[page, kh]
    for b in range(len(lens)):
        n = min(int(lens[b]), table.shape[1] * lay.P)
        cnt = starts[b + 1] - starts[b]
        if n <= 0 or cnt == 0:
            continue
        blocks = (n + lay.P - 1) // lay.P
        live = np.zeros(blocks * lay.P, bool)
        for kh in range(lay.Hk):
            c, s, z = (np.zeros((2, blocks * lay.P, D)) for _ in range(3))
            for i in range(blocks):
                pg = table[b, i]
                if 0 <= pg < cache.shape[0]:
                    live[i * lay.P:(i + 1) * lay.P] = True
                    cc, ss, zz = rec(pg, kh)
                    sl = slice(i * lay.P, (i + 1) * lay.P)
                    c[:, sl], s[:, sl], z[:, sl] = cc, ss, zz
            for r in range(cnt):
                t = starts[b] + r
                pos = int(lens[b]) - cnt + r
                ids = np.arange(max(0, pos - window + 1) if window else 0, min(pos + 1, n))
                ids = ids[live[ids]]
                if pos < 0 or len(ids) == 0:
                    continue
                k, v = (c[0, ids] - z[0, ids]) * s[0, ids], (c[1, ids] - z[1, ids]) * s[1, ids]
                pk, pv = s[0, ids] * (c[0, ids] + z[0, ids]), s[1, ids] * (c[1, ids] + z[1, ids])
                for h in range(kh * grp, (kh + 1) * grp):
                    sc = (k @ q[t, h]) * scale
                    m = sc.max()
                    e = np.exp(sc - m)
                    p = e / e.sum()
                    lse[t, h] = m + np.log(e.sum())
                    out[t, h] = p @ v
                    absv[t, h] = p @ np.abs(v)
                    cz[t, h] = p @ pv
                    dmax[t, h] = scale * (pk @ np.abs(q[t, h])).max()
                    keys[t, h] = len(ids)
                    smax[t, h] = s[1, ids].max()
    return out, lse, absv, cz, dmax, keys, smax
