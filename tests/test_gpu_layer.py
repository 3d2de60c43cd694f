"""GPU: the operators between a decoder layer's products (residual norm to 8-bit
rows, append to the paged 8-bit cache, attention over it) against the float64
oracle, through the public entry points."""
import numpy as np
import pytest

import oracle as O
from tests._helpers import say

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

U = 2.0 ** -24          # float32 unit roundoff
H = 2.0 ** -11          # fp16 unit roundoff


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemv_nibble_unpack_amd as G
    G.load()
    return G


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


# ------------------------------------------------------------------ norm
def check_norm(codes, scale, x, w, res, eps, kind, what):
    """scale within float32 rounding of max|y| / L; every code's value within half a
    code step of y / scale (plus float32 rounding), so ties may fall either way."""
    h, y = O.rmsnorm_rows(x, w, res, eps)
    K = x.shape[1]
    Lim = 127.0 if kind == 0 else 448.0
    s64 = np.abs(y).max(axis=1) / Lim
    # h, the sum of K squares (blocked: at most K/512 + 16 additions deep), root,
    # product and quotient
    rel = (K / 512 + 32) * U
    assert np.all(np.abs(scale - s64) <= rel * s64 + 1e-44), what
    v = O.decode_q8(codes.view(np.uint8), kind).astype(np.float64)
    live = s64 > 0
    assert np.all(v[~live] == 0)
    q = y[live] / s64[live, None]
    err = np.abs(v[live] - q)
    if kind == 0:
        step = np.full_like(q, 1.0)
    else:
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -6))) - 3)
    bad = err > 0.5 * step + 16 * U * np.abs(q) + 1e-30
    assert not bad.any(), f"{what}: {int(bad.sum())} codes off, worst {err[bad].max()}"
    assert np.all(np.abs(v).max(axis=1)[live] == Lim), what


@pytest.mark.parametrize("M,K", [(1, 8), (1, 4096), (3, 24), (5, 1000), (7, 1032), (2, 4096),
                                 (300, 3200), (3, 8640), (2, 11008), (2, 16384), (2, 16392),
                                 (1, 131056), (513, 128)])
@pytest.mark.parametrize("dt", [np.float16, np.float32])
@pytest.mark.parametrize("kind", [0, 1])
def test_norm(g, M, K, dt, kind):
    rng = np.random.default_rng(M * 1000 + K)
    x = (rng.standard_normal((M, K)) * np.exp(rng.standard_normal(K))).astype(dt)
    r = rng.standard_normal((M, K)).astype(dt)
    w = (1 + 0.2 * rng.standard_normal(K)).astype(dt)
    if M > 1:
        x[1] = 0
        r[1] = 0
    say("norm", M, K, dt.__name__, kind)
    for res in (r, None):
        codes, scale, h = g.add_rmsnorm_q8(dev(x), dev(w), None if res is None else dev(res),
                                           eps=1e-5, q_dtype=kind)
        check_norm(host(codes), host(scale), x, w, res, 1e-5, kind, (M, K, dt, kind))
        if res is not None:
            want = (x.astype(np.float32) + r.astype(np.float32)).astype(dt)
            assert np.array_equal(host(h), want)


def test_norm_in_place_and_stream(g):
    rng = np.random.default_rng(5)
    for K in (4096, 20000):
        x, r = (rng.standard_normal((9, K)).astype(np.float16) for _ in range(2))
        w = np.ones(K, np.float16)
        a = g.add_rmsnorm_q8(dev(x), dev(w), dev(r))
        s = torch.cuda.Stream()
        rd, xd, wd = dev(r), dev(x), dev(w)
        torch.cuda.synchronize()
        b = g.add_rmsnorm_q8(xd, wd, rd, residual_out=rd, stream=s)
        s.synchronize()
        assert b[2].data_ptr() == rd.data_ptr()
        for p, q in zip(a, b):
            assert torch.equal(p, q)
        xd2 = dev(x)
        c = g.add_rmsnorm_q8(xd2, wd, dev(r), residual_out=xd2,
                             out=(torch.empty_like(a[0]), torch.empty_like(a[1])))
        assert torch.equal(c[0], a[0]) and torch.equal(xd2, a[2])


@pytest.mark.parametrize("kind", [0, 1])
def test_norm_special_rows(g, kind):
    K = 512
    x = np.random.default_rng(1).standard_normal((6, K)).astype(np.float32)
    x[1, 7], x[2, 9] = np.nan, np.inf
    x[3] *= np.float32(1e-30)
    x[4] *= np.float32(1e-42)             # subnormal
    w = np.ones(K, np.float32)
    codes, scale, _ = (host(t) for t in g.add_rmsnorm_q8(dev(x), dev(w), eps=1e-5, q_dtype=kind))
    assert np.isnan(scale[1]) and np.isnan(scale[2])
    assert not codes[1].any() and not codes[2].any()
    ok = [0, 3, 5]
    check_norm(codes[ok], scale[ok], x[ok], w, None, 1e-5, kind, "special")
    Lim = 127.0 if kind == 0 else 448.0
    v = O.decode_q8(codes[4].view(np.uint8), kind)
    q = x[4].astype(np.float64) / np.abs(x[4].astype(np.float64)).max() * Lim
    assert np.abs(v).max() == Lim and np.all(np.abs(v - q) <= 0.5 * (1 if kind == 0 else 32) + 1e-3)


def test_norm_feeds_products(g):
    """The codes and scales are the rows that the INT8 and FP8 products take."""
    rng = np.random.default_rng(8)
    M, N, K = 20, 96, 256
    x, r = (rng.standard_normal((M, K)).astype(np.float16) for _ in range(2))
    w = (1 + 0.1 * rng.standard_normal(K)).astype(np.float16)
    W = (0.02 * rng.standard_normal((N, K))).astype(np.float32)
    _, y = O.rmsnorm_rows(x, w, r, 1e-5)
    codes, scale, _ = g.add_rmsnorm_q8(dev(x), dev(w), dev(r))
    Wq, ws, _ = g.quantize_pack_w4(dev(W))
    C = host(g.w4a8_gemm(codes, scale, g.prepack_w(g.W4_LAYOUT_W4A8, Wq, N, K), ws, N,
                         out_dtype=g.W4_OUT_F32)).astype(np.float64)
    q4, s4 = O.quantize_w4_sym(W)
    ref = y @ (q4 * s4[:, None].astype(np.float64)).T
    # half a code per activation
    lim = 0.5 * (np.abs(y).max(1) / 127)[:, None] * np.abs(q4 * s4[:, None]).sum(1)[None]
    assert np.all(np.abs(C - ref) <= lim * (1 + 1e-3) + 1e-6)
    codes, scale, _ = g.add_rmsnorm_q8(dev(x), dev(w), dev(r), q_dtype=g.W4_Q_F8)
    Wq, ws = g.quantize_f8(dev(W))
    C = host(g.f8f8_gemm(codes, scale, g.prepack_w(g.W4_LAYOUT_W8A8, Wq, N, K), ws, N,
                         out_dtype=g.W4_OUT_F32)).astype(np.float64)
    wv = O.e4m3_decode(host(Wq)) * host(ws)[:, None].astype(np.float64)
    ref = y @ wv.T
    step = np.maximum(np.abs(y) / 16, (np.abs(y).max(1) / 448)[:, None] * 2.0 ** -10)
    assert np.all(np.abs(C - ref) <= step @ np.abs(wv).T * (1 + 1e-3) + 1e-6)


# ------------------------------------------------------------------ cache
def rope_table(rows, rot, base=10000.0, stretch=1.0):
    a = (np.arange(rows)[:, None] / stretch) * base ** (-np.arange(rot // 2) / max(1, rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def page_tables(rng, lens, page, spare=3):
    """Scattered page numbers, -1 past each sequence's last page; the pool's size."""
    need = [-(-n // page) for n in lens]
    pool = sum(need) + spare
    ids = rng.permutation(pool)[:sum(need)]
    t = np.full((len(lens), max(1, max(need))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = ids[at:at + n]
        at += n
    return t, pool


def device_codes(cache, which):
    c = cache.codes[which]
    c = c if which == 0 else c.transpose(0, 1, 3, 2)
    return dev(np.ascontiguousarray(c).view(np.int8 if cache.kind == 0 else np.uint8))


def check_cache(cache, kc, vc, ks, vs, what):
    for which, (c, s) in enumerate(((kc, ks), (vc, vs))):
        got = host(c).view(np.uint8)
        got = got if which == 0 else got.transpose(0, 1, 3, 2)
        assert np.array_equal(host(s), cache.scale[which], equal_nan=True), (what, which, "scale")
        assert np.array_equal(got, cache.codes[which]), \
            (what, which, int((got != cache.codes[which]).sum()))


def append_call(g, cache_dev, rows, table, kv_len, news, tab, style, dt, strided, with_q=True,
                **more):
    """rows: (q, k, v) of all tokens; the call as a layer makes it."""
    q, k, v = rows
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if strided:      # slices of a fused projection's rows, with a gap at the row's end
        f = np.concatenate([q, k, v], 1).reshape(T, -1)
        f = dev(np.concatenate([f, np.zeros((T, 8), f.dtype)], 1))
        cut = np.cumsum([0, Hq * D, Hkv * D, Hkv * D])
        qd, kd, vd = (f[:, cut[i]:cut[i + 1]].unflatten(1, (-1, D)) for i in range(3))
    else:
        qd, kd, vd = dev(q), dev(k), dev(v)
    one = all(n == 1 for n in news)
    indptr = None if one else dev(np.concatenate([[0], np.cumsum(news)]).astype(np.int32))
    return g.rope_append_kv8(qd if with_q else None, kd, vd, *cache_dev, dev(table),
                             dev(np.asarray(kv_len, np.int32)), q_indptr=indptr,
                             max_q=max(1, max(news)), rope=None if tab is None else dev(tab),
                             style=style, **more)


APPENDS = [  # page, Hq, Hkv, D, rot, style, batches of new tokens per sequence
    (16, 4, 4, 128, 128, 0, [[17, 1, 33], [1, 1, 1], [5, 16, 1]]),
    (64, 8, 2, 64, 64, 1, [[100, 0, 64, 1], [1, 1, 1, 1], [3, 70, 0, 63]]),
    (32, 2, 1, 100, 100, 0, [[31, 2], [1, 1], [1, 1]]),
    (16, 5, 1, 100, 64, 1, [[15, 16, 40], [2, 3, 1]]),
    (128, 3, 3, 256, 128, 0, [[129, 250], [1, 1], [30, 2]]),
    (64, 2, 2, 80, 0, 0, [[64, 5], [1, 1]]),
    (32, 14, 2, 192, 96, 1, [[1], [1], [40]]),
    (16, 4, 2, 96, 4, 0, [[20, 20], [9, 1]]),
]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dt", [np.float16, np.float32])
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append(g, case, dt, kind):
    """Codes and scales bit for bit after each of several appends (prompt, single
    tokens, chunks; pages begun, filled and re-coded), queries to one rounding."""
    page, Hq, Hkv, D, rot, style, batches = APPENDS[case]
    rng = np.random.default_rng(100 + case)
    B = len(batches[0])
    lens = np.sum(batches, axis=0)
    table, pool = page_tables(rng, lens, page)
    dp = g.kv8_padded_dim(D)
    cache = O.PagedCache8(pool, page, Hkv, D, dp, kind)
    for c in cache.codes:                        # what an earlier owner left in the pages
        c[..., :D] = rng.integers(0, 0x70, c[..., :D].shape)
    cdev = (device_codes(cache, 0), device_codes(cache, 1), dev(cache.scale[0]), dev(cache.scale[1]))
    tab = rope_table(int(lens.max()) + 1, rot) if rot else None
    done = np.zeros(B, int)
    for step, news in enumerate(batches):
        say("append", case, dt.__name__, kind, "step", step)
        T = sum(news)
        # later tokens are larger, so that scales grow inside pages
        gain = 1.0 + step
        q, k, v = (gain * rng.standard_normal((T, h, D)) for h in (Hq, Hkv, Hkv))
        q, k, v = (a.astype(dt) for a in (q, k, v))
        kv_len = done + news
        got = append_call(g, cdev, (q, k, v), table, kv_len, news, tab, style, dt, step % 2 == 0)
        pos = np.concatenate([np.arange(d, d + n) for d, n in zip(done, news)])
        kr = O.rope_f32(k, tab, pos, rot, style)
        qr = O.rope_f32(q, tab, pos, rot, style)
        at = 0
        for b, n in enumerate(news):
            if n:
                cache.append((kr[at:at + n], v[at:at + n].astype(np.float32)), table[b], done[b])
            at += n
        assert np.array_equal(host(got), qr.astype(np.float16))
        check_cache(cache, *cdev, (case, dt, kind, step))
        done = kv_len


@pytest.mark.parametrize("kind", [0, 1])
def test_append_special_values(g, kind):
    """Zero rows, tiny and huge magnitudes, NaN and infinity, a poisoned page begun
    anew, queries left out, fp16 queries turned in place."""
    page, Hkv, D = 16, 2, 64
    table = np.array([[3, 1], [0, 2]], np.int32)
    cache = O.PagedCache8(4, page, Hkv, D, 64, kind)
    cdev = g.kv8_alloc(4, page, Hkv, D, q_dtype=kind)
    rng = np.random.default_rng(3)
    steps = [np.zeros((2, Hkv, D)), rng.standard_normal((2, Hkv, D)) * 1e-38,
             rng.standard_normal((2, Hkv, D)) * 1e30, rng.standard_normal((2, Hkv, D))]
    bad = rng.standard_normal((2, Hkv, D))
    bad[0, 0, 5], bad[1, 1, 6] = np.nan, -np.inf
    steps += [bad, rng.standard_normal((2, Hkv, D))]
    tab = rope_table(40, D)
    for i, a in enumerate(steps):
        a = a.astype(np.float32)
        append_call(g, cdev, (a, a, a), table, [i + 1, i + 1], [1, 1], tab, 0, np.float32, False,
                    with_q=False)
        with np.errstate(invalid="ignore"):
            kr = O.rope_f32(a, tab, np.array([i, i]), D, 0)
        for b in range(2):
            cache.append((kr[b:b + 1], a[b:b + 1]), table[b], i)
        check_cache(cache, *cdev, (kind, i))
    assert np.isnan(cache.scale[1][3, 0]) and np.isnan(cache.scale[1][0, 1])
    # the pages serve another sequence
    a = rng.standard_normal((2, Hkv, D)).astype(np.float16)
    qd = dev(a)
    out = g.rope_append_kv8(qd, dev(a), dev(a), *cdev, dev(table), dev(np.array([1, 1], np.int32)),
                            rope=dev(tab), q_out=qd)
    for b in range(2):
        cache.append((O.rope_f32(a[b:b + 1], tab, np.array([0]), D, 0), a[b:b + 1].astype(np.float32)),
                     table[b], 0)
    check_cache(cache, *cdev, "anew")
    assert out.data_ptr() == qd.data_ptr()
    assert np.array_equal(host(out), O.rope_f32(a, tab, np.array([0, 0]), D, 0).astype(np.float16))


def test_append_in_place_queries_over_pages(g):
    """fp16 queries turned in place, half layout (pairs far apart), many tokens."""
    rng = np.random.default_rng(4)
    T, Hq, D, page = 150, 6, 128, 64
    table = np.arange(3, dtype=np.int32)[None]
    cdev = g.kv8_alloc(3, page, 2, D)
    tab = rope_table(T, D, stretch=4.0)
    q = rng.standard_normal((T, Hq, D)).astype(np.float16)
    k = rng.standard_normal((T, 2, D)).astype(np.float16)
    qd = dev(q)
    g.rope_append_kv8(qd, dev(k), dev(k), *cdev, dev(table), dev(np.array([T], np.int32)),
                      q_indptr=dev(np.array([0, T], np.int32)), max_q=T, rope=dev(tab), q_out=qd)
    assert np.array_equal(host(qd), O.rope_f32(q, tab, np.arange(T), D, 0).astype(np.float16))


def test_append_skips_what_does_not_fit(g):
    """Sequences with contradicting lengths are left alone; a page number outside the
    pool skips that page; the others are served."""
    rng = np.random.default_rng(6)
    page, Hkv, D = 16, 1, 64
    news = [3, 3, 3, 3, 20, 3]
    table = np.array([[0, 1], [2, 3], [4, 5], [6, 7], [8, 99], [10, 11]], np.int32)
    kv_len = np.array([3, 33, 2, 40, 20, 19], np.int32)   # ok, past table, too few, past table, page 99, ok
    T = sum(news)
    a = rng.standard_normal((T, Hkv, D)).astype(np.float16)
    tab = rope_table(25, D)
    cache = O.PagedCache8(12, page, Hkv, D, 64, 0)
    cdev = g.kv8_alloc(12, page, Hkv, D)
    q_out = torch.full((T, Hkv, D), 7.0, dtype=torch.float16, device="cuda")
    append_call(g, cdev, (a, a, a), table, kv_len, news, tab, 0, np.float16, False, q_out=q_out)
    at = 0
    want = np.full((T, Hkv, D), 7.0, np.float16)
    for b, n in enumerate(news):
        if b in (0, 4, 5):
            start = int(kv_len[b]) - n
            kr = O.rope_f32(a[at:at + n], tab, np.arange(start, start + n), D, 0)
            want[at:at + n] = kr.astype(np.float16)
            cache.append((kr, a[at:at + n].astype(np.float32)), table[b], start)
        at += n
    check_cache(cache, *cdev, "skips")
    assert np.array_equal(host(q_out), want)
    # more new tokens than max_q, a table shorter than the positions: nothing is written
    before = [t.clone() for t in cdev]
    d = dev(a[:3])
    for kw in (dict(max_q=2, rope=dev(tab)), dict(max_q=3, rope=dev(tab[:2]))):
        g.rope_append_kv8(d, d, d, *cdev, dev(table[:1]), dev(np.array([3], np.int32)),
                          q_indptr=dev(np.array([0, 3], np.int32)), q_out=q_out[:3], **kw)
    # q_indptr outside the tokens, decreasing
    g.rope_append_kv8(d, d, d, *cdev, dev(table[:3]), dev(np.array([3, 3, 3], np.int32)),
                      q_indptr=dev(np.array([-1, 9, 5, 2], np.int32)), max_q=3, rope=dev(tab),
                      q_out=q_out[:3])
    for x, y in zip(before, cdev):
        assert torch.equal(x, y)
    assert np.array_equal(host(q_out), want)


def test_append_extreme_lengths(g):
    """Lengths and offsets at the ends of their type are refused by the kernel itself."""
    lo, hi = -2 ** 31, 2 ** 31 - 1
    cdev = g.kv8_alloc(4, 16, 1, 64)
    x = dev(np.ones((5, 1, 64), np.float16))
    before = [t.clone() for t in cdev]
    q_out = torch.full((5, 1, 64), 7.0, dtype=torch.float16, device="cuda")
    table = dev(np.zeros((1, 2), np.int32))
    for n in (lo, lo + 4, -1, hi):
        for ip in ([0, 5], [0, hi], [lo, 5], [3, lo], [hi, lo]):
            g.rope_append_kv8(x, x, x, *cdev, table, dev(np.array([n], np.int32)),
                              q_indptr=dev(np.array(ip, np.int64).astype(np.int32)), max_q=5,
                              q_out=q_out)
    for a, b in zip(before, cdev):
        assert torch.equal(a, b)
    assert (host(q_out) == 7.0).all()


# ------------------------------------------------------------------ attention
def random_cache(rng, lens, page, Hkv, D, dp, kind, spread=1.0):
    table, pool = page_tables(rng, lens, page)
    cache = O.PagedCache8(pool, page, Hkv, D, dp, kind)
    for which in range(2):
        c = cache.codes[which]
        if kind == 0:
            c[..., :D] = np.clip(np.rint(40 * rng.standard_normal(c[..., :D].shape)), -127, 127) \
                .astype(np.int8).view(np.uint8)
            one = 1 / 40
        else:
            c[..., :D] = O.e4m3_encode((60 * rng.standard_normal(c[..., :D].shape)).astype(np.float32))
            one = 1 / 64
        cache.scale[which][:] = (one * np.exp(spread * rng.standard_normal(cache.scale[which].shape)))
    return cache, table


def spoil_past_end(cache, table, lens):
    """What lies in pages past the sequences' lengths must not matter: E4M3 NaNs and
    the largest codes there, NaN scales in unused pages."""
    used = set()
    for b, n in enumerate(lens):
        for j in range(-(-n // cache.page)):
            used.add(int(table[b, j]))
            lead = n - j * cache.page
            if lead < cache.page:
                for c in cache.codes:
                    c[table[b, j], :, lead:] = 0x7F
    for pid in set(range(cache.codes[0].shape[0])) - used:
        for c, s in zip(cache.codes, cache.scale):
            c[pid] = 0xFF
            s[pid] = np.nan


def attn_bound(ref, absv, terms, n, D):
    """fp16 output rounding; fp16 weights (relative 2^-11, and 2^-25 absolute before
    the factor 2^10 is taken out); float32 score error of D products and the
    exponent's argument (twice: weight and sum); float32 sums over n tokens."""
    score = ((D + 16) * terms + 64)[:, None] * U
    sums = (n / 32 + 160) * U
    return H * np.abs(ref) + (H * (1 + H) + 2 * score + 2 * sums) * absv + 2.0 ** -24


def check_attention(g, rng, cache, table, lens, news, Hq, scale=None, strided=False, graph=False,
                    max_kv=None, **more):
    Hkv, D, page = cache.codes[0].shape[1], cache.dim, cache.page
    G, T = Hq // Hkv, sum(news)
    q = rng.standard_normal((T, Hq, D)).astype(np.float16)
    if strided:
        f = torch.full((T, Hq * D + 12), 3.0, dtype=torch.float16, device="cuda")
        qd = f[:, 4:4 + Hq * D].unflatten(1, (Hq, D))
        qd.copy_(dev(q))
    else:
        qd = dev(q)
    one = all(n == 1 for n in news)
    indptr = None if one else dev(np.concatenate([[0], np.cumsum(news)]).astype(np.int32))
    lse = torch.full((T, Hq), 9.0, dtype=torch.float32, device="cuda")
    args = (device_codes(cache, 0), device_codes(cache, 1), dev(cache.scale[0]), dev(cache.scale[1]),
            dev(table), dev(np.asarray(lens, np.int32)),
            max(1, max(lens)) if max_kv is None else max_kv)
    kw = dict(q_indptr=indptr, max_q=max(1, max(news)), scale=scale, lse=lse, **more)
    out = g.paged_attn_kv8(qd, *args, **kw)
    got, glse = host(out).astype(np.float64), host(lse).astype(np.float64)
    scale = D ** -0.5 if scale is None else scale
    at, worst = 0, 0.0
    for b, n in enumerate(news):
        for h in range(Hkv if n else 0):
            k, v = (cache.rows(w, table[b], lens[b], h) for w in range(2))
            qs = q[at:at + n, h * G:(h + 1) * G].reshape(n * G, D)
            limits = np.repeat(lens[b] - n + 1 + np.arange(n), G)
            ref, rl, absv, terms = O.attention_rows(qs, k, v, limits, scale)
            bound = attn_bound(ref, absv, terms, max(lens[b], 1), D)
            o = got[at:at + n, h * G:(h + 1) * G].reshape(n * G, D)
            err = np.abs(o - ref)
            assert np.all(err <= bound), (b, h, float((err - bound).max()), float((err / bound).max()))
            worst = max(worst, float((err / bound).max()))
            l = glse[at:at + n, h * G:(h + 1) * G].reshape(-1)
            empty = limits <= 0
            assert np.all(np.isneginf(l[empty])) and np.all(o[empty] == 0)
            tol = ((D + 16) * terms + 64) * U + (max(lens[b], 1) / 32 + 200) * U + 8 * U * np.abs(rl)
            assert np.all(np.abs(l - rl)[~empty] <= tol[~empty])
        at += n
    return out, worst


ATTN = [  # page, Hq, Hkv, D, lens, news
    (64, 4, 4, 128, [1], [1]),
    (64, 4, 4, 128, [517, 64, 63, 65, 1], [1] * 5),
    (16, 8, 2, 64, [1, 15, 16, 17, 300], [1] * 5),
    (32, 16, 1, 96, [1000, 33], [1, 1]),
    (128, 7, 7, 100, [130, 128, 127], [1] * 3),
    (16, 8, 8, 80, [257, 513], [1, 1]),
    (64, 40, 1, 128, [777, 2], [1, 1]),
    (16, 6, 2, 192, [511, 40], [1, 1]),
    (64, 4, 1, 256, [1200, 65], [1, 1]),
    (32, 5, 1, 4, [70], [1]),
    (64, 8, 2, 128, [300, 64, 5, 2], [5, 0, 5, 2]),
    (16, 12, 4, 64, [40, 700], [40, 33]),
    (32, 4, 4, 100, [129, 250, 7], [129, 100, 1]),
    (64, 10, 2, 128, [260, 200], [260, 131]),
    (128, 4, 2, 256, [300], [150]),
    (64, 2, 2, 192, [160, 90], [65, 90]),
    (16, 32, 1, 96, [90, 20], [30, 1]),
    (64, 4, 4, 128, [3000], [1]),
    (64, 8, 1, 64, [5000, 10], [2, 2]),
]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention(g, case, kind):
    page, Hq, Hkv, D, lens, news = ATTN[case]
    rng = np.random.default_rng(200 + case)
    cache, table = random_cache(rng, lens, page, Hkv, D, g.kv8_padded_dim(D), kind)
    spoil_past_end(cache, table, lens)
    say("attention", case, kind)
    _, w = check_attention(g, rng, cache, table, lens, news, Hq, strided=case % 2 == 1)
    say("attention", case, kind, "worst share of the bound", round(w, 3))


@pytest.mark.parametrize("kind", [0, 1])
def test_attention_empty_rows_and_bounds(g, kind):
    """Lengths of zero and below the new tokens, a bound far above the lengths, a
    sharp and a negative softmax scale."""
    rng = np.random.default_rng(31)
    lens, news = [0, 2, 5, 70], [1, 4, 5, 3]
    cache, table = random_cache(rng, [max(1, n) for n in lens], 16, 2, 64, 64, kind)
    spoil_past_end(cache, table, lens)
    check_attention(g, rng, cache, table, lens, news, 4)
    check_attention(g, rng, cache, table, lens, news, 4, max_kv=1 << 20)
    check_attention(g, rng, cache, table, lens, news, 4, scale=2.0)
    check_attention(g, rng, cache, table, lens, news, 4, scale=-0.3)
    check_attention(g, rng, cache, table, lens, news, 4, scale=0.0)
    # only empty sequences, one token each
    cache, table = random_cache(rng, [1, 1], 16, 2, 64, 64, kind)
    check_attention(g, rng, cache, table, [0, 0], [1, 1], 4)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("n", [1, 40])
def test_attention_scales_far_apart(g, kind, n):
    """Value scales over many magnitudes, zero among them; key scales of zero."""
    rng = np.random.default_rng(32)
    lens = [400, 333]
    cache, table = random_cache(rng, lens, 16, 2, 128, 128, kind)
    cache.scale[1][:] = np.float32(10.0) ** rng.integers(-8, 2, cache.scale[1].shape)
    cache.scale[1][::3] = 0
    cache.scale[0][::4] = 0
    check_attention(g, rng, cache, table, lens, [n, n], 4)
    cache.scale[1][:] = 0
    out, _ = check_attention(g, rng, cache, table, lens, [n, n], 4)
    assert not host(out).any()


@pytest.mark.parametrize("n", [3, 70])
def test_attention_nan_where_it_is_seen(g, n):
    """A poisoned page and a page number outside the pool reach the rows that see a
    token of it, and no other row."""
    rng = np.random.default_rng(33)
    page, Hq, Hkv, D = 16, 4, 2, 64
    lens, news = [160 + n, 150], [n, 1]
    for what in ("k", "v", "table"):
        cache, table = random_cache(rng, lens, page, Hkv, D, 64, 0)
        j = (lens[0] - 1) // page                 # the last page of sequence 0
        if what == "table":
            table[0, j] = 10 ** 6
        else:
            cache.scale["kv".index(what)][table[0, j], 1] = np.nan
        T = sum(news)
        q = rng.standard_normal((T, Hq, D)).astype(np.float16)
        out = host(g.paged_attn_kv8(
            dev(q), device_codes(cache, 0), device_codes(cache, 1), dev(cache.scale[0]),
            dev(cache.scale[1]), dev(table), dev(np.array(lens, np.int32)), max(lens),
            q_indptr=dev(np.array([0, n, n + 1], np.int32)), max_q=n))
        pos = lens[0] - n + np.arange(n)
        sees = np.concatenate([pos >= j * page, [False]])
        want = np.zeros((T, Hq), bool)
        want[sees] = True
        if what != "table":
            want[:, :Hq // Hkv] = False
        nan = np.isnan(out)
        assert np.array_equal(nan.any(2), want), what
        assert np.array_equal(nan.all(2), want), what


def test_attention_lengths_that_do_not_fit(g):
    rng = np.random.default_rng(34)
    lens = [20, 20, 20, 20]
    cache, table = random_cache(rng, lens, 16, 1, 64, 64, 0)
    q = dev(rng.standard_normal((4, 2, 64)).astype(np.float16))
    cd = (device_codes(cache, 0), device_codes(cache, 1), dev(cache.scale[0]), dev(cache.scale[1]),
          dev(table))
    kv = dev(np.array([20, 33, -1, 21], np.int32))       # ok, past the table, negative, above max_kv
    out = host(g.paged_attn_kv8(q, *cd, kv, 20))
    assert np.isfinite(out[0]).all() and np.isnan(out[1:]).all()
    # more new tokens than max_q: the first max_q rows; q_indptr outside: untouched
    keep = torch.full((4, 2, 64), 5.0, dtype=torch.float16, device="cuda")
    kv = dev(np.array([20, 20, 20, 20], np.int32))
    out = host(g.paged_attn_kv8(q, *cd, kv, 20, q_indptr=dev(np.array([0, 3, 4, 2, 9], np.int32)),
                                max_q=2, out=keep))
    assert np.isnan(out[:2]).all() and (out[2] == 5.0).all() and np.isfinite(out[3]).all()


@pytest.mark.parametrize("max_q", [5, 100])
def test_attention_extreme_lengths(g, max_q):
    rng = np.random.default_rng(37)
    lo, hi = -2 ** 31, 2 ** 31 - 1
    cache, table = random_cache(rng, [20], 16, 1, 64, 64, 1)
    cd = (device_codes(cache, 0), device_codes(cache, 1), dev(cache.scale[0]), dev(cache.scale[1]),
          dev(table))
    q = dev(np.ones((5, 1, 64), np.float16))
    for n in (lo, -1, hi):
        out = host(g.paged_attn_kv8(q, *cd, dev(np.array([n], np.int32)), 20,
                                    q_indptr=dev(np.array([0, 5], np.int32)), max_q=max_q))
        assert np.isnan(out).all()
    for ip in ([0, hi], [lo, 5], [3, lo], [hi, lo], [4, 4]):
        keep = torch.full((5, 1, 64), 5.0, dtype=torch.float16, device="cuda")
        g.paged_attn_kv8(q, *cd, dev(np.array([20], np.int32)), 20, max_q=max_q, out=keep,
                         q_indptr=dev(np.array(ip, np.int64).astype(np.int32)))
        assert (host(keep) == 5.0).all(), ip


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("n", [33, 129, 300])
def test_attention_many_rows_split(g, kind, n):
    """Chunks of long contexts: row tiles alone and in pairs, split over blocks."""
    rng = np.random.default_rng(38)
    lens = [5000, 2600, n]
    cache, table = random_cache(rng, lens, 32, 1, 128, 128, kind)
    spoil_past_end(cache, table, lens)
    assert g.paged_attn_kv8_workspace_bytes(3, n + 40, n, 5000, 1, 1, 128) > 0
    _, w = check_attention(g, rng, cache, table, lens, [n, 35, 5], 1)
    say("split", kind, n, "worst share of the bound", round(w, 3))
    a, _ = check_attention(g, np.random.default_rng(1), cache, table, lens, [n, 35, 5], 1)
    b, _ = check_attention(g, np.random.default_rng(1), cache, table, lens, [n, 35, 5], 1)
    assert torch.equal(a, b)


@pytest.mark.parametrize("batch", [2, 64, 65])
def test_attention_many_sequences(g, batch):
    """Tiled attention of batches in any order of lengths, equal lengths among them."""
    rng = np.random.default_rng(39)
    news = [150 if b == batch // 2 else int(rng.integers(0, 4)) for b in range(batch)]
    lens = [max(n, int(rng.choice([0, 1, 40, 40, 200, 333]))) for n in news]
    cache, table = random_cache(rng, lens, 16, 1, 64, 64, 0)
    spoil_past_end(cache, table, lens)
    _, w = check_attention(g, rng, cache, table, lens, news, 2)
    say("sequences", batch, "worst share of the bound", round(w, 3))


@pytest.mark.parametrize("n", [1, 4])
def test_attention_split_repeats_bitwise_and_shares_workspace(g, n):
    """Long sequences are split over blocks: the same bits call after call, on another
    stream, and with a workspace that other shapes and products used in between."""
    rng = np.random.default_rng(35)
    lens = [9000, 70, 4097]
    cache, table = random_cache(rng, lens, 64, 2, 128, 128, 0)
    ws = g.Workspace()
    q = dev(rng.standard_normal((3 * n, 8, 128)).astype(np.float16))
    args = (device_codes(cache, 0), device_codes(cache, 1), dev(cache.scale[0]), dev(cache.scale[1]),
            dev(table), dev(np.asarray(lens, np.int32)), max(lens))
    kw = dict(q_indptr=dev(np.array([0, n, 2 * n, 3 * n], np.int32)), max_q=n)
    assert g.paged_attn_kv8_workspace_bytes(3, 3 * n, n, 9000, 8, 2, 128) > 0
    first = g.paged_attn_kv8(q, *args, **kw)
    W = dev((0.02 * rng.standard_normal((16, 131056))).astype(np.float32))
    codes = torch.randint(-1, 2, (16, 131056), dtype=torch.int8, device="cuda")
    Wp = g.prepack_w(g.W4_LAYOUT_W2A8, g.quantize_pack_w2(codes), 16, 131056)
    s16 = g.ternary_scale_f16(W)
    A = dev(rng.standard_normal((1, 131056)).astype(np.float16))
    Aq, sa, _ = g.quantize_a8(A)
    ref = g.w2a8_gemm(Aq, sa, Wp, s16, 16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(4):
        assert torch.equal(g.w2a8_gemm(Aq, sa, Wp, s16, 16, workspace=ws), ref)
        assert torch.equal(g.paged_attn_kv8(q, *args, workspace=ws, **kw), first)
        if i % 2:
            r = g.paged_attn_kv8(q, *args, workspace=ws, stream=side, **kw)
            side.synchronize()
            assert torch.equal(r, first)
    torch.cuda.synchronize()
    assert not ws.buf[:16384].any()
    check_attention(g, rng, cache, table, lens, [n] * 3, 8, workspace=ws)


def test_attention_far_pages(g):
    """Page offsets past 32 bits."""
    rng = np.random.default_rng(36)
    page, Hkv, D, dp = 64, 16, 128, 128
    pool = (1 << 32) // (page * Hkv * dp) + 40            # 4.3 GB of keys, as much of values
    kc = torch.zeros(pool, Hkv, page, dp, dtype=torch.int8, device="cuda")
    vc = torch.zeros(pool, Hkv, dp, page, dtype=torch.int8, device="cuda")
    ks = torch.zeros(pool, Hkv, device="cuda")
    vs = torch.zeros(pool, Hkv, device="cuda")
    lens = [200, 90]
    table = np.array([[pool - 1, 3, pool - 7, pool - 2], [pool - 3, 5, -1, -1]], np.int32)
    small = O.PagedCache8(8, page, Hkv, D, dp, 0)
    local = np.array([[0, 1, 2, 3], [4, 5, -1, -1]], np.int32)
    k, v = (rng.standard_normal((290, Hkv, D)).astype(np.float16) for _ in range(2))
    q = rng.standard_normal((290, Hkv, D)).astype(np.float16)
    indptr = dev(np.array([0, 200, 290], np.int32))
    kvl = dev(np.array(lens, np.int32))
    g.rope_append_kv8(None, dev(k), dev(v), kc, vc, ks, vs, dev(table), kvl, q_indptr=indptr,
                      max_q=200)
    for b, (a, z) in enumerate(((0, 200), (200, 290))):
        small.append((k[a:z].astype(np.float32), v[a:z].astype(np.float32)), local[b], 0)
    ids = torch.from_numpy(np.concatenate([table[0], table[1, :2]]).astype(np.int64)).cuda()
    check_cache(small, *[torch.cat([t[ids], torch.zeros_like(t[:2])]) for t in (kc, vc, ks, vs)],
                "far pages")
    for n in (1, 64):
        rows = np.concatenate([q[200 - n:200], q[290 - n:290]])
        ip = dev(np.array([0, n, 2 * n], np.int32))
        out = host(g.paged_attn_kv8(dev(rows), kc, vc, ks, vs, dev(table), kvl, 200, q_indptr=ip,
                                    max_q=n)).astype(np.float64)
        for b in range(2):
            for h in (0, 15):
                kk, vv = (small.rows(w, local[b], lens[b], h) for w in range(2))
                ref, _, absv, terms = O.attention_rows(rows[b * n:(b + 1) * n, h], kk, vv,
                                                       lens[b] - n + 1 + np.arange(n), D ** -0.5)
                assert np.all(np.abs(out[b * n:(b + 1) * n, h] - ref) <=
                              attn_bound(ref, absv, terms, lens[b], D))


# ------------------------------------------------------------------ together
def test_step_graph_replays(g):
    """Norm, append and attention of a decode step in one graph: lengths advance on the
    device between replays, every replay equals the eager calls, bit for bit."""
    rng = np.random.default_rng(41)
    B, Hq, Hkv, D, page, steps = 3, 8, 2, 128, 16, 6
    K = (Hq + 2 * Hkv) * D
    start = np.array([30, 15, 63], np.int32)
    table, pool = page_tables(rng, start + steps, page)
    tab = dev(rope_table(128, D))
    xs = [dev(rng.standard_normal((B, K)).astype(np.float16)) for _ in range(steps)]
    w = dev(np.ones(K, np.float16))

    def state():
        c = g.kv8_alloc(pool, page, Hkv, D)
        k = dev(np.random.default_rng(1).standard_normal((int(start.sum()), Hkv, D)).astype(np.float16))
        g.rope_append_kv8(None, k, k, *c, dev(table), dev(start),
                          q_indptr=dev(np.concatenate([[0], np.cumsum(start)]).astype(np.int32)),
                          max_q=int(start.max()), rope=tab)
        f16 = dict(dtype=torch.float16, device="cuda")
        return dict(c=c, x=torch.empty(B, K, **f16), res=torch.zeros(B, K, **f16), len=dev(start.copy()),
                    codes=torch.empty(B, K, dtype=torch.int8, device="cuda"),
                    sc=torch.empty(B, device="cuda"), q=torch.empty(B, Hq, D, **f16),
                    o=torch.empty(B, Hq, D, **f16), t=dev(table),
                    ws=torch.zeros(g.W4_ATTN_WORKSPACE_MAX, dtype=torch.uint8, device="cuda"))

    def step(s):
        g.add_rmsnorm_q8(s["x"], w, s["res"], residual_out=s["res"], out=(s["codes"], s["sc"]))
        qkv = s["x"].view(B, -1, D)
        g.rope_append_kv8(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], *s["c"], s["t"],
                          s["len"], rope=tab, q_out=s["q"])
        g.paged_attn_kv8(s["q"], *s["c"], s["t"], s["len"], 128 * page, workspace=s["ws"], out=s["o"])

    eager, replayed = state(), state()
    stream = torch.cuda.Stream()
    graph = g.StepGraph(stream)
    torch.cuda.synchronize()
    with graph.capture():
        step(replayed)
    assert graph.kernel_nodes() == 3
    for x in xs:
        for s in (eager, replayed):
            s["x"].copy_(x)
            s["len"].add_(1)
        step(eager)
        torch.cuda.synchronize()
        graph.launch()
        stream.synchronize()
        for name in ("o", "q", "codes", "sc", "res"):
            assert torch.equal(eager[name], replayed[name]), name
        for a, b in zip(eager["c"], replayed["c"]):
            assert torch.equal(a, b)
    graph.close()
