"""Edges of the serving operators on the GPU: sizes at which a call is laid out in another way than
its neighbours, values at the ends of their types, work on other streams."""
import numpy as np
import pytest
import torch

import weight_only_quantization_act_amd as awq
from tests.gpu_util import requires_gpu, say
from tests.kv4_ref import attention
from tests.test_gpu_kv4 import Case, _check, _compare, _within

pytestmark = [pytest.mark.gpu, requires_gpu]

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("T,M,K", [(32, 128, 2040), (16, 16384, 4095), (333, 640, 3063), (2, 16500, 4085),
                                   (40, 300, 1023), (100, 1000, 5 * 1024 - 1)])
def test_linear_stays_in_its_workspace(T, M, K):
    """Columns that are no multiple of 16 and end just below another division of K: the result is the
    two calls' and the bytes behind the workspace stay as they were."""
    say(f"int8 linear workspace T={T} M={M} K={K}")
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(T, K, generator=g, device="cuda").half()
    W = (torch.randn(M, K, generator=g, device="cuda") * 0.02).half()
    wq, ws = awq.awq_int8_quantize(W)
    need = awq.awq_int8_linear_workspace_bytes(T, M, K)
    guard = 2 * T * M * 4 * 8 + 4096               # more than any division's sums
    buf = torch.full((need + guard,), 0x5A, dtype=torch.uint8, device="cuda")
    y = awq.awq_int8_linear(x, wq, ws, workspace=buf[:need])
    assert (buf[need:] == 0x5A).all()
    xq, xs = awq.awq_int8_quantize(x)
    assert torch.equal(y, awq.awq_int8_matmul(xq, xs, wq, ws))
    acc = xq.cpu().numpy().astype(np.float64) @ wq.cpu().numpy().astype(np.float64).T  # exact
    want = (acc.astype(np.float32) * xs.cpu().numpy()[:, None] * ws.cpu().numpy()).astype(np.float16)
    assert np.array_equal(y.cpu().numpy(), want)


@pytest.mark.parametrize("n,Hk,grp", [(64, 8, 8), (2048, 1, 4), (40, 2, 1)])
def test_window_with_a_loose_bound(n, Hk, grp):
    """A bound on the lengths so loose that only the window lets the tiles be counted: the keys are
    divided, into the workspace that the query named, and the result is that of a tight bound."""
    lens = [int(x) for x in np.random.default_rng(n).integers(0, 300 if n > 100 else 2000, n)]
    c = Case(64, Hk, 16, 64, 1, lens, [1] * n, seed=n)
    c.fill()
    q = torch.randn(n, Hk * grp, 64, device="cuda").half()
    for window, max_len in ((8192, 1 << 30), (1 << 20, 1 << 30), ((1 << 63) - 1, 1 << 30), (8192, 1 << 24),
                            (50, 1 << 30)):
        say(f"kv4 window={window} max_len={max_len} n={n}")
        need = awq.awq_kv4_attention_workspace_bytes(n, n, Hk * grp, c.cfg, 1, max_len)
        buf = torch.full((need + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
        out, lse = awq.awq_kv4_attention(q, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=1,
                                         max_len=max_len, window=window, workspace=buf[:need])
        assert (buf[need:] == 0x5A).all()
        _compare(c, q, out, lse, None, min(window, 1 << 20), where=(n, window, max_len))


# How a call is laid out: sequences, key heads, rows a sequence, bound on the lengths.
FORMS = {"eight waves": (5, 2, 1, 0), "four waves": (300, 1, 2, 0), "divided": (5, 2, 1, 9000),
         "divided, many parts": (2, 1, 3, 100000), "prompt": (3, 2, 30, 0), "prompt, split": (1, 1, 30, 0)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_nan_reaches_the_rows_that_see_it(form, dtype):
    """NaN is never taken for a key that is not there: a query row with a NaN, a key that holds
    one and is alone in its tile, keys that all hold one.  Rows without keys stay rows without keys."""
    say(f"kv4 nan {form} {dtype}")
    n, Hk, news, bound = FORMS[form]
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(news, 400, n)]
    lens[0] = 0 if news == 1 else lens[0]            # a row without keys
    lens[-1] = 33 if news < 30 else 1025
    c = Case(128, Hk, 16, 64, 1, lens, [news] * n, dtype, seed=n)
    bound = bound or max(lens)

    def run(spoil_keys, spoil_q):
        k, v = c.kv(sum(lens))
        starts = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device="cuda")
        spoil_keys(k, starts)
        awq.awq_kv4_append(k, v, c.cache, c.dtable, c.dlens, starts, c.cfg)
        q = torch.randn(n * news, 3 * Hk, 128, device="cuda").to(c.dt)
        spoil_q(q)
        out, lse = awq.awq_kv4_attention(q, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=news,
                                         max_len=bound)
        o, ls = out.isnan(), lse.isnan()
        assert torch.equal(o.all(-1), o.any(-1)) and torch.equal(o.all(-1), ls)
        if lens[0] == 0:
            assert not out[0].any() and torch.isneginf(lse[0]).all()
        return ls.cpu().numpy()

    keys = np.repeat(np.array(lens) > 0, news)[:, None]

    def nothing(*_):
        pass
    assert not run(nothing, nothing).any()
    bad = np.zeros((n * news, 3 * Hk), bool)          # every third row, one head
    bad[::3, 1] = True

    def spoil_q(q):
        q[::3, 1, 77] = float("nan")
    assert np.array_equal(run(nothing, spoil_q), bad & keys)
    # the last token of the last sequence, first key head: seen by the last row only
    bad[:] = False
    bad[-1, :3] = True

    def last_key(k, starts):
        k[-1, 0, 3] = float("nan")
    assert np.array_equal(run(last_key, nothing), bad)
    bad[:] = False
    bad[:, :3] = True

    def all_keys(k, starts):
        k[:, 0, 100] = float("nan")
    assert np.array_equal(run(all_keys, nothing), bad & keys)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("news", [1, 40])
def test_queries_at_the_ends_of_their_type(dtype, news):
    """Query rows from the type's subnormals to its largest values, with a scale that brings the
    scores back to about one: each row is scaled exactly, so the model's bound holds as ever."""
    c = Case(64, 2, 32, 64, 1, (300, 77), (news, news), dtype, seed=news)
    c.fill()
    info = torch.finfo(c.dt)
    lo, hi = (-22, 15) if dtype == "fp16" else (-131, 127)
    q0 = torch.randn(2 * news, 4, 64, device="cuda")
    q0 /= q0.abs().amax(-1, keepdim=True)               # largest magnitude 1
    for exp in sorted({lo, lo + 3, -126 if lo < -126 else lo, -110, -100, -93, -92, 0, 92, 108, 115, 116, 117,
                       hi - 1, hi}):
        if not lo <= exp <= hi:
            continue
        say(f"kv4 queries of 2^{exp} {dtype} rows={news}")
        q = (q0.double() * 2.0 ** exp).clamp(float(info.min), float(info.max)).to(c.dt)
        assert q.isfinite().all() and (q != 0).any()
        _check(c, q, 2.0 ** min(-3 - exp, 127), 0, where=(exp, dtype, news))


@pytest.mark.parametrize("news", [1, 40])
def test_scales_at_the_ends(news):
    """Scales down to fp32's least subnormal: the scores vanish and masked keys still count nothing.
    Up to its largest: rows whose scores are 0 are averages still."""
    c = Case(128, 2, 32, 64, 1, (300, 77, 0), (news, news, 1), "bf16", seed=news)
    c.fill()
    q = torch.randn(2 * news + 1, 4, 128, device="cuda").bfloat16()
    for scale in (2.0 ** -149, 2.0 ** -140, 2.0 ** -126, 2.0 ** -118, 2.0 ** -100):
        say(f"kv4 scale {scale} rows={news}")
        for x in (q, q * 2.0 ** 100, q * 2.0 ** -100):
            _check(c, x, scale, 0, where=(scale, news))
            _check(c, x, scale, 50, where=(scale, news, "window"))
    for scale in (1e30, 2.9e38, float(np.finfo(np.float32).max)):
        say(f"kv4 scale {scale} rows={news}")
        _check(c, q * 0, scale, 0, where=(scale, news))
        _check(c, q * 0, scale, 50, where=(scale, news, "window"))


@pytest.mark.parametrize("form", FORMS)
def test_infinite_queries(form):
    """A query row with an infinity is NaN whatever the signs of the codes it meets: keys of one sign
    make all its scores +infinity or all -infinity."""
    say(f"kv4 infinite queries {form}")
    n, Hk, news, bound = FORMS[form]
    lens = [int(x) for x in np.random.default_rng(n).integers(news, 400, n)]
    lens[0] = 0 if news == 1 else lens[0]
    for zp in (0, 1):
        c = Case(64, Hk, 16, 32, zp, lens, [news] * n, "bf16", seed=n)
        k, v = c.kv(sum(lens))
        k = -k.abs() - 1
        starts = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device="cuda")
        awq.awq_kv4_append(k, v, c.cache, c.dtable, c.dlens, starts, c.cfg)
        q = torch.randn(n * news, 3 * Hk, 64, device="cuda").bfloat16()
        q[::2, 0, 5], q[1::2, 1, 63] = float("inf"), float("-inf")
        out, lse = awq.awq_kv4_attention(q, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=news,
                                         max_len=bound or max(lens))
        keys = torch.from_numpy(np.repeat(np.array(lens) > 0, news))[:, None].cuda()
        want = ~torch.isfinite(q).all(-1) & keys
        assert torch.equal(out.isnan().all(-1), want) and torch.equal(out.isnan().any(-1), want)
        assert torch.equal(lse.isnan(), want)
        assert torch.equal(torch.isneginf(lse), (~keys).expand_as(lse)) and not out[~keys[:, 0]].any()


@pytest.mark.parametrize("D,g", [(128, 64), (128, 128), (64, 32), (64, 64)])
@pytest.mark.parametrize("spoil", ["nan", "huge"])
def test_values_that_do_not_count_cost_no_precision(D, g, spoil):
    """Small values beside a token whose value is NaN or huge: rows that the mask keeps from it meet
    the bound of their own values, and so do, beside a NaN, the channels of other groups."""
    rng = np.random.default_rng(D + g)
    for lens, news, window, at in (((300,), 1, 20, (-21,)),            # just before the window, in its tile
                                   ((300, 90), 3, 40, (-45, -44)),     # several rows, divided below
                                   ((200, 150), 40, 0, (-1,)),         # prompt: later than all rows but one
                                   ((500,), 90, 64, (-155, -30))):     # before some windows, inside others
        say(f"kv4 values beside {spoil} D={D} g={g} news={news} window={window}")
        n = len(lens)
        c = Case(D, 1, 16, g, 1, lens, [news] * n, "bf16", seed=news)
        k, v = c.kv(sum(lens))
        v = v * 2.0 ** -13
        ends = np.cumsum(lens)
        rows = [int(e + a) for e in ends for a in at]
        fill = float("nan") if spoil == "nan" else 6.0e5              # a step of about 40000
        v[rows, 0, 1] = fill
        starts = torch.tensor(np.concatenate(([0], ends)), dtype=torch.int32, device="cuda")
        awq.awq_kv4_append(k, v, c.cache, c.dtable, c.dlens, starts, c.cfg)
        q = torch.from_numpy(rng.standard_normal((n * news, 3, D))).to(c.dt).cuda()
        pos = np.concatenate([np.arange(x - news, x) for x in lens])
        own = np.repeat(ends - np.array(lens), news)                   # first row of the sequence in k, v
        hit = np.zeros(n * news, bool)
        for r in rows:
            p = r - own
            hit |= (p >= 0) & (p <= pos) & (pos - p < (window or 1 << 30))
        assert (~hit).any()
        ref = attention(c.lay, q.double().cpu().numpy(), c.cache.cpu().numpy(), c.table, c.lens, c.starts,
                        D ** -0.5, window)
        if spoil == "nan":
            # channels of the other groups in all rows: their sums never touch the NaN
            vc = v.clone()
            vc[rows, 0, :g] = v[0, 0, :g]
            clean = Case(D, 1, 16, g, 1, lens, [news] * n, "bf16", seed=news)
            awq.awq_kv4_append(k, vc, clean.cache, clean.dtable, clean.dlens, starts, clean.cfg)
            ref2 = attention(c.lay, q.double().cpu().numpy(), clean.cache.cpu().numpy(), clean.table,
                             c.lens, c.starts, D ** -0.5, window)
        for bound in (max(lens), 9000):
            out, lse = awq.awq_kv4_attention(q, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=news,
                                             max_len=bound, window=window)
            keep = torch.from_numpy(~hit).cuda()
            _within(c.lay, out[keep], lse[keep], [x[~hit] for x in ref], (news, window, bound))
            if spoil == "nan":
                assert out[~keep][..., :g].isnan().all()
                if g < D:
                    want, wl, absv, cz, dmax, keys, smax = ref2
                    _within(c.lay, out[..., g:], lse, (want[..., g:], wl, absv[..., g:], cz[..., g:], dmax, keys,
                                                       smax), (news, window, bound, "other groups"))


def test_more_rows_than_a_grid_dimension():
    """2^24 rows and more, a block of 256 threads each: the codes of every part by itself."""
    say("int8 rows 2^24 + 3")
    R, K = (1 << 24) + 3, 16
    A = torch.empty((R, K), dtype=torch.float16, device="cuda").normal_()
    q, st = awq.awq_int8_quantize(A)
    for a in range(0, R, 1 << 22):
        qa, sa = awq.awq_int8_quantize(A[a:a + (1 << 22)])
        assert torch.equal(q[a:a + (1 << 22)], qa) and torch.equal(st[a:a + (1 << 22)], sa), a
    want = A[-3:].float().abs().amax(1) / torch.full((3,), 127.0, device="cuda")
    assert torch.equal(st[-3:], want)
    wq, ws = awq.awq_int8_quantize(torch.randn(3, K, device="cuda").half())
    y = awq.awq_int8_linear(A, wq, ws)
    assert torch.equal(y[-1000:], awq.awq_int8_linear(A[-1000:], wq, ws))
    assert torch.equal(y[:1000], awq.awq_int8_linear(A[:1000], wq, ws))


def test_more_blocks_than_a_grid_dimension_write_the_cache():
    """65535 sequences on 160 key heads, more than 2^24 blocks of 256 threads: the few that have a new
    token write and read back what they would by themselves."""
    say("kv4 store, 65535 sequences x 160 heads")
    n, Hk = 65535, 160
    cfg = awq.awq_kv4_config(64, Hk, 16, 64, 1)
    seqs = [0, 1, 777, 40000, 52429, 65533, 65534]
    news = np.zeros(n, np.int64)
    news[seqs] = 2
    lens = np.where(news > 0, 9, 0)
    table = np.full((n, 1), -1, np.int32)
    table[seqs, 0] = np.arange(len(seqs))
    T = int(news.sum())
    k, v = torch.randn(2, T + 3, Hk, 64, device="cuda").half()

    def run(pick):
        def ints(x):
            return torch.from_numpy(np.ascontiguousarray(x)).to(torch.int32).cuda()
        cache = awq.awq_kv4_cache(len(seqs), cfg)
        args = (cache, ints(table[pick]), ints(lens[pick]),
                ints(np.concatenate(([0], np.cumsum(news[pick])))), cfg)
        awq.awq_kv4_append(k, v, *args)
        return (cache, *awq.awq_kv4_read(*args, T + 3))
    all_of, few = run(np.arange(n)), run(np.array(seqs))
    for a, b in zip(all_of, few):
        assert torch.equal(a, b)
    assert few[1][:T].any(-1).all() and not few[1][T:].any()


def test_more_rows_than_a_grid_dimension_are_joined():
    """2^24 rows and more of which the sequence has four, its keys divided over many parts: the join, a
    block a row, reaches them all and writes no other."""
    say("kv4 join, 2^24 + 5 rows")
    T, news = (1 << 24) + 5, 4
    c = Case(64, 1, 64, 64, 1, (9000,), (news,), seed=1)
    c.fill()
    out = torch.full((T, 1, 64), 7.0, dtype=torch.float16, device="cuda")
    q = torch.randn(1, 1, 64, device="cuda").half().expand(T, 1, 64)
    # an empty sequence holds the rows before the last four
    table = torch.cat([c.dtable * 0 - 1, c.dtable])
    lens = torch.tensor([0, 9000], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, T - news, T], dtype=torch.int32, device="cuda")
    got, lse = awq.awq_kv4_attention(q, c.cache, table, lens, starts, c.cfg, max_q=news, max_len=9000, out=out)
    want, wl = awq.awq_kv4_attention(q[:news], c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=news,
                                     max_len=9000)
    assert got is out
    assert torch.allclose(got[-news:].float(), want.float(), rtol=2.0 ** -10, atol=2.0 ** -9)
    assert torch.allclose(lse[-news:], wl, rtol=0, atol=2.0 ** -17)
    assert not got[:news].any() and torch.isneginf(lse[:news]).all()
    assert (got[news:-news] == 7).all()


def test_more_outputs_than_a_grid_dimension():
    """One token through 2^28 outputs and more, a block of 512 threads for every 32: each part as it is
    by itself."""
    say("int8 linear, 2^28 + 40 outputs")
    M, K = (1 << 28) + 40, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    wq = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand(M, generator=g, device="cuda")
    x = torch.randn(1, K, generator=g, device="cuda").half()
    y = torch.full((1, M), float("nan"), device="cuda").half()
    awq.awq_int8_linear(x, wq, ws, out=y)
    for a in range(0, M, 1 << 26):
        part = slice(a, min(a + (1 << 26), M))
        assert torch.equal(y[:, part], awq.awq_int8_linear(x, wq[part], ws[part])), a
    xq, xs = awq.awq_int8_quantize(x)
    want = (xq.double() @ wq[-5:].double().t()).float() * xs[:, None] * ws[-5:]
    assert torch.equal(y[:, -5:], want.half())


@pytest.mark.parametrize("news", [1, 50])
def test_cache_operators_on_another_stream(news):
    """Work follows the given stream: what is made on a side stream is read after it, and a workspace and
    outputs that the call allocates belong to that stream."""
    say(f"kv4 side stream rows={news}")
    lens = (2000, 300, 77)
    c = Case(128, 2, 16, 64, 1, lens, [news] * 3, seed=news)
    c.fill()
    ref = Case(128, 2, 16, 64, 1, lens, [news] * 3, seed=news)
    ref.cache.copy_(c.cache)
    T = 3 * news
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    for rep in range(4):
        with torch.cuda.stream(side):
            for _ in range(4):
                big = torch.mm(big, big).clamp_(-1, 1)       # keeps the stream busy
            x = torch.randn(3, T, 8, 128, device="cuda").half() + big[0, 0].half() * 0
        awq.awq_kv4_append(x[0, :, :2], x[1, :, :2], c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, stream=side)
        k, v = awq.awq_kv4_read(c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, T, stream=side)
        out, lse = awq.awq_kv4_attention(x[2], c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=news,
                                         max_len=2000, stream=side)
        side.synchronize()
        awq.awq_kv4_append(x[0, :, :2], x[1, :, :2], ref.cache, c.dtable, c.dlens, c.dstarts, c.cfg)
        k2, v2 = awq.awq_kv4_read(ref.cache, c.dtable, c.dlens, c.dstarts, c.cfg, T)
        o2, l2 = awq.awq_kv4_attention(x[2], ref.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=news,
                                       max_len=2000)
        torch.cuda.synchronize()
        assert torch.equal(c.cache, ref.cache) and torch.equal(k, k2) and torch.equal(v, v2), rep
        assert torch.equal(out, o2) and torch.equal(lse, l2), rep


@pytest.mark.parametrize("form", FORMS)
def test_keys_of_infinite_step(form):
    """Keys so large (bf16) that their step is infinite in fp16 are NaN to the rows that see them, whatever
    the sign of what they give, and nothing to the others."""
    say(f"kv4 keys of infinite step {form}")
    n, Hk, news, bound = FORMS[form]
    lens = [int(x) for x in np.random.default_rng(n).integers(news + 1, 400, n)]
    for sign in (1, -1):
        c = Case(64, Hk, 16, 32, 1, lens, [news] * n, "bf16", seed=n)
        k, v = c.kv(sum(lens))
        ends = np.cumsum(lens)
        at = [int(e) - 1 - b % 3 * (news // 2) for b, e in enumerate(ends)]   # one key a sequence, head 0
        k[at, 0, 32:] = sign * 4.0e6
        starts = torch.tensor(np.concatenate(([0], ends)), dtype=torch.int32, device="cuda")
        awq.awq_kv4_append(k, v, c.cache, c.dtable, c.dlens, starts, c.cfg)
        q = torch.rand(n * news, 3 * Hk, 64, device="cuda").bfloat16() + 0.1
        out, lse = awq.awq_kv4_attention(q, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=news,
                                         max_len=bound or max(lens))
        row = np.concatenate([np.arange(e - news, e) for e in ends])          # the rows' own tokens
        want = np.zeros((n * news, 3 * Hk), bool)
        want[:, :3] = (row >= np.repeat(at, news))[:, None]
        assert np.array_equal(lse.isnan().cpu().numpy(), want), (sign, form)
        assert np.array_equal(out.isnan().all(-1).cpu().numpy(), want)
        assert np.array_equal(out.isnan().any(-1).cpu().numpy(), want)
