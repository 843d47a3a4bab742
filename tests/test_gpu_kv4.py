"""The 4-bit key/value cache and its attention on the GPU against a 64-bit numpy model that
looks every value up at its own byte.

Bars, derived from the kernels' arithmetic:
  - cache bytes: defined by single IEEE fp32 operations, equal bit for bit; bytes of other
    tokens untouched;
  - read-back: (code - zero) * step is one fp32 rounding, then one to the output type;
  - attention: q is exact in its operand (but for parts 2^-24 below the row's largest, absolute
    2^-25 of it).  A score is an fp32 sum over head_dim products and the group terms: its error
    is at most e_s = (head_dim + 64) 2^-24 scale sum_i |q_i| step (c_i + z) in the exponent
    (largest over the row's keys), which counts twice in out (weight and normaliser) and once
    in lse; exp2 and its argument add 2^-21 + 2^-23 |exponent range|, taken as 2^-19; the
    weights are rounded to fp16 (2^-11 relative each, and 2^-38 of the largest step for what
    lies in fp16's subnormals); fp32 sums over n keys of weight (c + z) step add at most
    (n / 8 + 64) 2^-24 of sum p step (c + z).  Then one ulp of the output type.
"""
import numpy as np
import pytest
import torch

import weight_only_quantization_act_amd as awq
from tests.gpu_util import requires_gpu, say
from tests.kv4_ref import Layout, attention

pytestmark = [pytest.mark.gpu, requires_gpu]

F64 = np.float64
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _ulp(v, dtype):
    bits, emin = (10, -14) if dtype == torch.float16 else (7, -126)
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** emin)))
    return 2.0 ** (np.maximum(e, emin) - bits)


class Case:
    """A cache with sequences of the given lengths, rows for the last `news` tokens of each."""

    def __init__(self, D, Hk, P, g, zp, lens, news, dtype="fp16", seed=0, spare=3, extra_blocks=2):
        self.lay = Layout(D, Hk, P, g, zp)
        self.cfg = awq.awq_kv4_config(D, Hk, P, g, zp)
        assert awq.awq_kv4_record_bytes(self.cfg) == self.lay.record
        self.dt = DT[dtype]
        self.rng = np.random.default_rng(seed)
        self.lens, self.news = list(lens), list(news)
        self.starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
        blocks = [max(0, (n + P - 1) // P) for n in lens]
        width = max(1, max(blocks)) + extra_blocks
        self.n_pages = sum(blocks) + spare
        perm = self.rng.permutation(self.n_pages)
        self.table = np.full((len(lens), width), -1, np.int32)   # unused entries: no page
        at = 0
        for b, n in enumerate(blocks):
            self.table[b, :n] = perm[at:at + n]
            at += n
        # what no token was written to holds anything: random bytes, so NaN and infinite steps
        self.cache = torch.from_numpy(self.rng.integers(
            0, 256, (self.n_pages, Hk, self.lay.record), dtype=np.uint8)).cuda()
        self.dtable, self.dstarts = torch.from_numpy(self.table).cuda(), torch.from_numpy(self.starts).cuda()
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def kv(self, T, spread=1.0):
        x = torch.from_numpy(self.rng.standard_normal((2, T, self.lay.Hk, self.lay.D)) * spread)
        x[..., ::13] *= 8
        return x[0].to(self.dt).cuda(), x[1].to(self.dt).cuda()

    def fill(self, spread=1.0):
        """Write every token of every sequence through the library."""
        n = [max(0, x) for x in self.lens]
        starts = torch.tensor(np.concatenate(([0], np.cumsum(n))), dtype=torch.int32, device="cuda")
        k, v = self.kv(sum(n), spread)
        awq.awq_kv4_append(k, v, self.cache, self.dtable, self.dlens, starts, self.cfg)
        return k, v


LAYOUTS = [(64, 64), (64, 32), (128, 128), (128, 64), (128, 32)]


@pytest.mark.parametrize("D,g", LAYOUTS)
@pytest.mark.parametrize("zp", [0, 1])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_bytes_and_read(D, g, zp, dtype):
    """Cache bytes equal the model's; nothing else changes; the read-back is the values."""
    for P, Hk, lens, news in ((16, 3, (1, 37, 0, 16), (1, 20, 1, 5)), (64, 1, (130, 3), (67, 3)),
                              (256, 2, (5, -1, 257), (9, 2, 1))):
        say(f"kv4 append D={D} g={g} P={P} zp={zp} {dtype}")
        c = Case(D, Hk, P, g, zp, lens, news, dtype, seed=P + D)
        T = int(c.starts[-1])
        k, v = c.kv(T + 2)                                     # two rows past the last sequence
        k[0, 0, :g] = 0                                        # a group of zeros
        v[T // 2, Hk - 1] = 3.25                               # equal values
        k[T // 2, 0, D - 1] = float("nan")
        v[T // 3, 0, 0] = float("inf")
        want = c.cache.cpu().numpy().copy()
        kn, vn = k.float().cpu().numpy(), v.float().cpu().numpy()
        exists = np.zeros(T + 2, bool)
        place = {}
        for b in range(len(lens)):
            for r in range(news[b]):
                pos = lens[b] - news[b] + r
                t = c.starts[b] + r
                if pos < 0:
                    continue
                exists[t] = True
                for h in range(Hk):
                    rec = want[c.table[b, pos // P], h]
                    c.lay.write(rec, pos % P, 0, kn[t, h])
                    c.lay.write(rec, pos % P, 1, vn[t, h])
                    place[t, h] = (c.table[b, pos // P], pos % P)
        awq.awq_kv4_append(k, v, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg)
        got = c.cache.cpu().numpy()
        assert np.array_equal(got, want), (np.argwhere(got != want)[:4], D, g, P)
        ko, vo = awq.awq_kv4_read(c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, T + 2, dtype=c.dt)
        for side, o in ((0, ko), (1, vo)):
            o = o.float().cpu().numpy()
            assert not o[~exists].any()
            for (t, h), (pg, p) in place.items():
                code, st, z = (x[side, p] for x in c.lay.decode(want[pg, h]))
                w = torch.from_numpy(((code - z) * st)).float().to(c.dt).float().numpy()
                assert np.array_equal(o[t, h], w, equal_nan=True), (t, h, side)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("zp", [0, 1])
def test_append_steps_at_the_ends(dtype, zp):
    """Ranges from the type's subnormals to its largest values, each with every magnitude of its
    16-bit values, exact halves of the step, steps of all mantissa bits, and ranges that overflow:
    the bytes are the model's."""
    lay = Layout(64, 1, 16, 32, zp)
    info = torch.finfo(DT[dtype])
    rng = np.random.default_rng(5)
    n = 256
    c = Case(64, 1, 16, 32, zp, (n,), (n,), dtype, seed=1)
    x = rng.standard_normal((n, 1, 64))
    exps = np.linspace(np.log2(float(info.tiny)) - 9, np.log2(float(info.max)) - 1, n)
    x = np.clip(x, -2, 2) / 2 * (2.0 ** exps)[:, None, None]
    x[10] = np.arange(64)[None] - 20                       # ties: range 31 or 43 over 15 steps
    x[11] = (np.arange(64)[None] % 16) * 0.5               # step 1/2: quotients are integers
    x[12] = (np.arange(64)[None] % 31 - 15) * 0.25
    x[13, 0, :32], x[13, 0, 32:] = float(info.max), float(info.min)
    x[14, 0, 0], x[14, 0, 1] = float(info.max), float(info.min)
    k = torch.from_numpy(x).to(c.dt).cuda()
    # steps whose mantissa is all ones or next to it, where a range of the type's values gives one
    vals = torch.arange(0, 32768, device="cuda", dtype=torch.int32).to(torch.int16).view(c.dt)
    vals = vals[torch.isfinite(vals)].float().cpu().numpy()
    st = (vals / np.float32(15 if zp else 7)).astype(np.float32)
    pick = vals[np.argsort(-(st.view(np.uint32) & 0x7fffff).astype(np.int64))[:n]]
    v = rng.uniform(-1, 1, (n, 1, 64)) * pick[:, None, None] * (0 if zp else 1)
    if zp:
        v = rng.uniform(0, 1, (n, 1, 64)) * pick[:, None, None]
    v[:, 0, 5] = pick
    v[:, 0, 40] = pick
    v = torch.from_numpy(v).to(c.dt).cuda()
    want = c.cache.cpu().numpy().copy()
    kn, vn = k.float().cpu().numpy(), v.float().cpu().numpy()
    for t in range(n):
        rec = want[c.table[0, t // 16], 0]
        lay.write(rec, t % 16, 0, kn[t, 0])
        lay.write(rec, t % 16, 1, vn[t, 0])
    awq.awq_kv4_append(k, v, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg)
    got = c.cache.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]


def test_append_strided_and_lost_pages():
    """Views into a fused projection; table entries that name no page drop their tokens."""
    c = Case(128, 2, 32, 64, 1, (100, 40), (100, 40), seed=3)
    T = 140
    qkv = torch.randn(T, 7, 2, 128, device="cuda").half()
    k, v = qkv[:, 5], qkv[:, 6]
    c2 = Case(128, 2, 32, 64, 1, (100, 40), (100, 40), seed=3)
    awq.awq_kv4_append(k, v, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg)
    awq.awq_kv4_append(k.contiguous(), v.contiguous(), c2.cache, c2.dtable, c2.dlens, c2.dstarts, c2.cfg)
    assert torch.equal(c.cache, c2.cache)
    # heads outermost: token stride 128, head stride T * 128
    kh = k.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    c3 = Case(128, 2, 32, 64, 1, (100, 40), (100, 40), seed=3)
    awq.awq_kv4_append(kh, v, c3.cache, c3.dtable, c3.dlens, c3.dstarts, c3.cfg)
    assert torch.equal(c.cache, c3.cache)
    bad = c.dtable.clone()
    bad[0, 1], bad[1, 0] = -5, c.n_pages
    c4 = Case(128, 2, 32, 64, 1, (100, 40), (100, 40), seed=3)
    before = c4.cache.clone()
    awq.awq_kv4_append(k, v, c4.cache, bad, c4.dlens, c4.dstarts, c4.cfg)
    lost = [int(c.table[0, 1]), int(c.table[1, 0])]
    for p in range(c.n_pages):
        assert torch.equal(c4.cache[p], before[p] if p in lost else c.cache[p]), p
    ko, _ = awq.awq_kv4_read(c4.cache, bad, c4.dlens, c4.dstarts, c4.cfg, T)
    assert not ko[32:64].any() and not ko[100:132].any() and ko[64:100].any()


def _check(c, q, scale, window, max_q=None, max_len=None, out=None, where=""):
    got, lse = awq.awq_kv4_attention(q, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg,
                                     max_q=max(c.news) if max_q is None else max_q,
                                     max_len=max(max(c.lens), 0) if max_len is None else max_len,
                                     scale=scale, window=window)
    _compare(c, q, got, lse, scale, window, where)
    return got, lse


def _compare(c, q, got, lse, scale, window, where=""):
    sc = c.lay.D ** -0.5 if scale is None else scale
    T = int(c.starts[-1])
    ref = attention(c.lay, q[:T].double().cpu().numpy(), c.cache.cpu().numpy(), c.table, c.lens,
                    c.starts, sc, window)
    _within(c.lay, got[:T], lse[:T], ref, where)


def _within(lay, got, lse, ref, where=""):
    want, wl, absv, cz, dmax, keys, smax = ref
    g, ls = got.double().cpu().numpy(), lse.double().cpu().numpy()
    es = (lay.D + 64) * 2.0 ** -24 * dmax
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(ls), empty), (where, ls, wl)
    el = np.zeros_like(ls)
    el[~empty] = np.abs(ls[~empty] - wl[~empty])
    assert (el <= es + 2.0 ** -19 + 2.0 ** -22 * np.abs(np.where(empty, 0, wl))).all(), (where, el.max())
    n = keys[..., None]
    E = (absv * (2 * es[..., None] + 2.0 ** -19 + 2.0 ** -11) + (n / 8 + 64) * 2.0 ** -24 * cz
         + n * 15 * 2.0 ** -38 * smax[..., None])
    bound = E + _ulp(np.abs(want) + E, got.dtype)
    err = np.abs(g - want)
    bad = ~(err <= bound)
    assert not bad.any(), (where, int(bad.sum()), np.argwhere(bad)[:3], g[bad][:3], want[bad][:3],
                           bound[bad][:3])
    assert not g[empty].any()


@pytest.mark.parametrize("D,g", LAYOUTS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_decode(D, g, dtype):
    """One row a sequence: lengths around the tiles and pages, an idle slot, every group size."""
    for P, Hk, grp, lens in ((16, 2, 4, (1, 15, 16, 17, 31, 32, 33, 0, 100)), (64, 1, 1, (63, 64, 65, 200)),
                             (128, 2, 16, (129, 300)), (32, 1, 7, (700, -3, 9)), (256, 3, 3, (255, 257))):
        say(f"kv4 decode D={D} g={g} P={P} heads={Hk}x{grp} {dtype}")
        c = Case(D, Hk, P, g, (D + g) // 32 % 2, lens, [1] * len(lens), dtype, seed=D + P)
        c.fill()
        q = torch.randn(len(lens), Hk * grp, D, device="cuda").to(c.dt)
        _check(c, q, None, 0, where=(P, Hk, grp))
        _check(c, q, 0.3, 20, where=(P, Hk, grp, "window"))


@pytest.mark.parametrize("D,g", LAYOUTS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rows(D, g, dtype):
    """Several rows a sequence, with and without earlier context, ragged, one row before the
    first token, more query heads than a tile has columns."""
    for P, Hk, grp, lens, news in ((16, 2, 4, (70, 5, 33, 1, 300), (70, 8, 2, 1, 17)),
                                   (32, 1, 20, (40, 150), (3, 40)), (64, 2, 1, (200, 64, 100), (130, 64, 1)),
                                   (128, 1, 8, (500,), (260,)), (16, 1, 2, (0, 9, 2), (3, 0, 2))):
        for window in (0, 1, 25):
            say(f"kv4 rows D={D} g={g} P={P} heads={Hk}x{grp} window={window} {dtype}")
            c = Case(D, Hk, P, g, 1, lens, news, dtype, seed=D + P + window)
            c.fill()
            q = torch.randn(int(c.starts[-1]), Hk * grp, D, device="cuda").to(c.dt)
            _check(c, q, None, window, where=(P, Hk, grp, window))


@pytest.mark.parametrize("D,g", LAYOUTS)
def test_sequences_dealt_out(D, g):
    """More sequences than lanes, of very different lengths: a block does parts of several, some
    without rows, without keys or before their first token."""
    rng = np.random.default_rng(D + g)
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(300), 150))]
    news = [int(x) for x in rng.integers(0, 4, 150)]
    lens[3], lens[5], lens[64], lens[100], lens[149] = 0, -2, 2500, 1, 1300
    news[3], news[5], news[7], news[64], news[149] = 1, 3, 0, 3, 1
    for n in (150, 65, 4):
        c = Case(D, 2, 16 if n == 65 else 64, g, 1, lens[:n], news[:n], "fp16", seed=n)
        c.fill()
        q = torch.randn(int(c.starts[-1]), 10, D, device="cuda").half()
        for window in (0, 700, 3):
            say(f"kv4 dealt out D={D} g={g} n={n} window={window}")
            a, la = _check(c, q, None, window, max_len=6000, where=(n, window))
            b, lb = awq.awq_kv4_attention(q, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=max(c.news),
                                          max_len=6000, window=window)
            assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("D,g", LAYOUTS)
def test_many_short_sequences(D, g):
    """A block a sequence, no second launch."""
    rng = np.random.default_rng(D + g)
    lens = [int(x) for x in rng.integers(-1, 90, 600)]
    news = [int(x) for x in rng.integers(0, 3, 600)]
    c = Case(D, 1, 32, g, 0, lens, news, "bf16", seed=g)
    c.fill()
    q = torch.randn(int(c.starts[-1]), 8, D, device="cuda").bfloat16()
    assert awq.awq_kv4_attention_workspace_bytes(len(q), 600, 8, c.cfg, 2, 1000) == 0
    for window in (0, 33):
        say(f"kv4 short D={D} g={g} window={window}")
        _check(c, q, None, window, max_q=2, max_len=1000, where=window)


@pytest.mark.parametrize("news", [1, 3, 40])
def test_long_context_splits(news):
    """Few sequences and many keys: the keys are split over blocks and joined."""
    c = Case(128, 2, 64, 128, 1, (5003, 700), (news, news), seed=news)
    c.fill()
    q = torch.randn(2 * news, 8, 128, device="cuda").half()
    assert awq.awq_kv4_attention_workspace_bytes(2 * news, 2, 8, c.cfg, news, 5003) > 0
    a, la = _check(c, q, None, 0)
    b, lb = _check(c, q, None, 0)
    assert torch.equal(a, b) and torch.equal(la, lb)                  # bit for bit again
    _check(c, q, None, 1000)
    _check(c, q, None, 0, max_len=100000)                             # a loose bound


def test_score_and_value_ranges():
    """Large scores (one key takes all the weight), tiny and huge value steps side by side, tiny
    and huge queries, rising scores (the running maximum changes in every tile)."""
    for D, g, dtype in ((128, 128, "fp16"), (64, 32, "bf16")):
        say(f"kv4 ranges D={D} g={g} {dtype}")
        n = 400
        c = Case(D, 1, 16, g, 1, (n,), (1,), dtype, seed=5)
        rng = c.rng
        q0 = rng.standard_normal(D)
        ramp = np.linspace(0, 1, n)[:, None]
        for kscale, vscale, qs in ((ramp * 3, 1.0, 1.0), (1.0, np.exp(rng.uniform(-9, 9, (n, 1))), 1.0),
                                   (1.0, 2.0 ** -12, 2.0 ** -9), (20.0, 1.0, 40.0), (1.0, 1.0, 2.0 ** -14),
                                   (-ramp * 3, np.exp(np.linspace(8, -8, n))[:, None], 1.0)):
            k = torch.from_numpy((q0 * kscale + rng.standard_normal((n, D)) * 0.3)[:, None]).to(c.dt).cuda()
            v = torch.from_numpy((rng.standard_normal((n, D)) * vscale)[:, None]).to(c.dt).cuda()
            st = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            awq.awq_kv4_append(k, v, c.cache, c.dtable, c.dlens, st, c.cfg)
            q = torch.from_numpy(np.stack([q0 * qs, -q0 * qs, np.zeros(D), rng.standard_normal(D) * qs])[None])
            _check(c, q.to(c.dt).cuda(), None, 0, where=(D, qs))


def test_nan_keys_stay_where_they_are_seen():
    """A token whose key or value holds a NaN or an infinity spoils the rows that see it, and no
    other: not earlier rows of the same tile, not other heads, not rows past its window."""
    for dtype in ("fp16", "bf16"):
        c = Case(128, 2, 16, 64, 1, (90,), (90,), dtype, seed=8)
        k, v = c.kv(90)
        k[41, 0, 5] = float("nan")
        v[50, 0, 100] = float("inf")
        awq.awq_kv4_append(k, v, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg)
        q = torch.randn(90, 6, 128, device="cuda").to(c.dt)
        for window in (0, 10):
            out, lse = awq.awq_kv4_attention(q, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=90,
                                             max_len=90, window=window)
            o, ls = out.isnan().cpu().numpy(), lse.isnan().cpu().numpy()
            rows = np.arange(90)
            seek = (rows >= 41) & ((rows < 51) if window else True)
            seev = (rows >= 50) & ((rows < 60) if window else True)
            assert np.array_equal(ls[:, :3], np.repeat(seek[:, None], 3, 1))
            assert not o[:, 3:].any() and not ls[:, 3:].any()
            assert o[seek][:, :3].all()
            assert o[seev][:, :3, 64:].all()                          # the infinite group
            assert not o[~seek & ~seev][:, :3].any()
            assert not o[seev & ~seek][:, :3, :64].any()              # the value's other group
            # and the finite rows are the numbers that they would be without those tokens
            c2 = Case(128, 2, 16, 64, 1, (90,), (90,), dtype, seed=8)
            k2, v2 = k.clone(), v.clone()
            k2[41, 0, 5], v2[50, 0, 100] = 0, 0
            awq.awq_kv4_append(k2, v2, c2.cache, c2.dtable, c2.dlens, c2.dstarts, c2.cfg)
            o2, l2 = awq.awq_kv4_attention(q, c2.cache, c2.dtable, c2.dlens, c2.dstarts, c2.cfg, max_q=90,
                                           max_len=90, window=window)
            _compare(c2, q, o2, l2, None, window)
            early = rows < 41
            el = torch.from_numpy(early).cuda()
            assert (out[el].float() - o2[el].float()).abs().max() <= 2.0 ** -9 * o2[el].float().abs().max()


def test_bounds_strides_and_lost_pages():
    """Rows beyond max_q are left alone, keys beyond max_len and on no page are masked, strided
    queries, an output given by the caller, rows past the last sequence."""
    c = Case(128, 2, 32, 128, 1, (200, 90), (5, 2), seed=4)
    c.fill()
    base = torch.randn(9, 3, 8, 128, device="cuda").half()
    q = base[:, 1]
    out = torch.full((9, 8, 128), 5.0, dtype=torch.float16, device="cuda")
    got, lse = awq.awq_kv4_attention(q, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=5, max_len=200,
                                     out=out)
    assert got is out and (out[7:] == 5).all()
    _compare(c, q, out, lse, None, 0)
    hm = q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    got2, _ = awq.awq_kv4_attention(hm, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=5, max_len=200)
    assert torch.equal(got2[:7], out[:7])
    out.fill_(5)
    awq.awq_kv4_attention(q, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=2, max_len=200, out=out)
    assert (out[2:5] == 5).all()
    out[2:5] = got2[2:5]   # (another bound may sum in another order: the rows meet the bar again)
    _compare(c, q, out, lse, None, 0)
    # a lost page in the middle of sequence 0: its keys do not exist
    tab = c.table.copy()
    c.table[0, 2] = c.n_pages + 7
    c.dtable[0, 2] = c.n_pages + 7
    _check(c, q, None, 0)
    c.table[0, 3] = -1
    c.dtable[0, 3] = -1
    _check(c, q, None, 40)
    c.table, c.dtable = tab, torch.from_numpy(tab).cuda()
    # keys beyond the caller's bound: rows 0 .. 4, at positions 195 and up, see keys 0 .. 149
    got, lse = awq.awq_kv4_attention(q, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=5, max_len=150)
    for r in range(5):
        ref = attention(c.lay, q[r:r + 1].double().cpu().numpy(), c.cache.cpu().numpy(), c.table[:1],
                        [150], np.array([0, 1]), 128 ** -0.5, 0)
        _within(c.lay, got[r:r + 1], lse[r:r + 1], ref, r)


def test_fewer_rows_than_the_starts_say():
    """q_start may point past the rows that q has: those rows do not exist."""
    for lens, news, T in (((40, 90), (5, 7), 9), ((40, 90, 3), (50, 40, 1), 70), ((3000, 2500), (2, 3), 4)):
        c = Case(128, 2, 32, 64, 1, lens, news, seed=T)
        c.fill()
        n = sum(news)
        q = torch.randn(n, 4, 128, device="cuda").half()
        a, la = awq.awq_kv4_attention(q, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=max(news),
                                      max_len=max(lens))
        out = torch.full((n, 4, 128), 7.0, device="cuda").half()
        b, lb = awq.awq_kv4_attention(q[:T], c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=max(news),
                                      max_len=max(lens), out=out[:T])
        assert (out[T:] == 7).all()
        # the same keys in the same order, but for where a division of the work cuts them
        assert torch.allclose(b.float(), a[:T].float(), rtol=2.0 ** -10, atol=2.0 ** -9)
        assert torch.allclose(lb, la[:T], rtol=0, atol=2.0 ** -17)


def test_offsets_beyond_32_bits():
    """Pages whose bytes lie past 4 GiB of the cache."""
    cfg = awq.awq_kv4_config(128, 8, 256, 128, 1)
    lay = Layout(128, 8, 256, 128, 1)
    n_pages = (5 << 30) // (8 * lay.record)
    cache = torch.zeros((n_pages, 8, lay.record), dtype=torch.uint8, device="cuda")
    pages = [n_pages - 1, 0, n_pages - 2]
    c = Case(128, 8, 256, 128, 1, (600,), (600,), seed=2)
    k, v = c.kv(600)
    small = Case(128, 8, 256, 128, 1, (600,), (600,), seed=2)
    awq.awq_kv4_append(k, v, small.cache, small.dtable, small.dlens, small.dstarts, cfg)
    table = torch.tensor([pages], dtype=torch.int32, device="cuda")
    awq.awq_kv4_append(k, v, cache, table, c.dlens, c.dstarts, cfg)
    ka, va = awq.awq_kv4_read(cache, table, c.dlens, c.dstarts, cfg, 600)
    kb, vb = awq.awq_kv4_read(small.cache, small.dtable, c.dlens, c.dstarts, cfg, 600)
    assert torch.equal(ka, kb) and torch.equal(va, vb)
    for news in (1, 50):
        st = torch.tensor([0, news], dtype=torch.int32, device="cuda")
        q = torch.randn(news, 32, 128, device="cuda").half()
        a, la = awq.awq_kv4_attention(q, cache, table, c.dlens, st, cfg, max_q=news, max_len=600)
        b, lb = awq.awq_kv4_attention(q, small.cache, small.dtable, c.dlens, st, cfg, max_q=news, max_len=600)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_graph_replays_follow_the_lengths():
    """A decode step (append, attention) captured once and replayed while the lengths grow:
    every replay equals the eager step, with eager work between the replays."""
    c = Case(128, 2, 16, 64, 1, (700, 20, 333), (1, 1, 1), seed=6, extra_blocks=4, spare=20)
    used = int((c.table >= 0).sum())
    free = [p for p in range(c.n_pages) if p not in set(c.table[c.table >= 0].tolist())]
    for b in range(3):
        row = c.table[b]
        for i in range(len(row)):
            if row[i] < 0 and free:
                row[i] = free.pop()
    assert used > 0
    c.dtable = torch.from_numpy(c.table).cuda()
    c.fill()
    k, v = c.kv(3)
    q = torch.randn(3, 8, 128, device="cuda").half()
    eager_cache = c.cache.clone()
    ws = torch.empty(awq.awq_kv4_attention_workspace_bytes(3, 3, 8, c.cfg, 1, 760) + 256,
                     dtype=torch.uint8, device="cuda")

    def step(cache, lens):
        awq.awq_kv4_append(k, v, cache, c.dtable, lens, c.dstarts, c.cfg)
        return awq.awq_kv4_attention(q, cache, c.dtable, lens, c.dstarts, c.cfg, max_q=1, max_len=760,
                                     workspace=ws)
    lens = c.dlens.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c.cache.clone(), lens)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = step(c.cache, lens)
    for rep in range(4):
        lens += 1
        k.normal_()
        v.normal_()
        q.normal_()
        g.replay()
        torch.cuda.synchronize()
        o2, l2 = step(eager_cache, lens)
        assert torch.equal(out, o2) and torch.equal(lse, l2), rep
        assert torch.equal(c.cache, eager_cache)


def test_refusals_of_the_binding():
    c = Case(128, 2, 32, 64, 1, (40,), (1,))
    q = torch.randn(1, 4, 128, device="cuda").half()
    args = (c.cache, c.dtable, c.dlens, c.dstarts, c.cfg)
    kw = dict(max_q=1, max_len=40)
    with pytest.raises(TypeError):
        awq.awq_kv4_attention(q.float(), *args, **kw)
    with pytest.raises(ValueError):
        awq.awq_kv4_attention(q[..., :64], *args, **kw)
    with pytest.raises(ValueError):
        awq.awq_kv4_attention(q, c.cache[:, :1].contiguous(), *args[1:], **kw)
    with pytest.raises(TypeError):
        awq.awq_kv4_attention(q, c.cache, c.dtable.long(), *args[2:], **kw)
    with pytest.raises(ValueError):
        awq.awq_kv4_attention(q, c.cache, c.dtable, c.dlens, c.dlens, c.cfg, **kw)
    with pytest.raises(awq.AwqError):
        awq.awq_kv4_attention(q, *args, scale=0.0, **kw)
    with pytest.raises(awq.AwqError):
        awq.awq_kv4_attention(torch.randn(1, 3, 128, device="cuda").half(), *args, **kw)
    with pytest.raises(awq.AwqError):
        awq.awq_kv4_attention(q, *args, window=-1, **kw)
    k = torch.randn(1, 2, 128, device="cuda").half()
    with pytest.raises(TypeError):
        awq.awq_kv4_append(k, k.bfloat16(), *args)
    with pytest.raises(ValueError):
        awq.awq_kv4_append(k, torch.cat([k, k]), *args)
    with pytest.raises(awq.AwqError):   # rows not 16-byte aligned
        awq.awq_kv4_append(torch.randn(300, device="cuda").half()[1:257].view(1, 2, 128), k, *args)
    with pytest.raises(ValueError):
        awq.awq_kv4_cache(4, awq.awq_kv4_config(96, 2, 32, 32, 1))
