"""GPU: the decoder-layer operators at the edges of their arguments' ranges, against
the oracle."""
import numpy as np
import pytest

import oracle as O
from tests._helpers import say
from tests.test_gpu_layer import (append_call, attn_bound, check_cache, check_norm, dev, device_codes, g,  # noqa: F401
                                  host, rope_table)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


# one wave, four, eight and sixteen a row, rows read twice
WIDTHS = [8, 1000, 4096, 8192, 12288, 16384, 20000]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dt", [np.float16, np.float32])
def test_norm_zero_rows_without_eps(g, dt, kind):  # noqa: F811
    """eps = 0: a row of zeros gets scale 0 and codes 0, its neighbours what they get alone."""
    rng = np.random.default_rng(1)
    for K in WIDTHS:
        x = rng.standard_normal((6, K)).astype(dt)
        w = (1 + 0.2 * rng.standard_normal(K)).astype(dt)
        x[1] = x[4] = 0
        r = -x
        r[[0, 2, 3, 5]] = 0
        r[1] = x[1]
        for res in (None, r):
            codes, scale, _ = (host(t) for t in g.add_rmsnorm_q8(
                dev(x), dev(w), None if res is None else dev(res), eps=0.0, q_dtype=kind))
            say("zero rows", K, dt.__name__, kind, scale[[1, 4]])
            assert not scale[[1, 4]].any() and not codes[[1, 4]].any()
            live = [0, 2, 3, 5]
            check_norm(codes[live], scale[live], x[live], w, None if res is None else res[live], 0.0,
                       kind, (K, dt, kind))
        # zeros after the weights: the same, whatever the root
        z = host(g.add_rmsnorm_q8(dev(x), dev(np.zeros(K, dt)), eps=0.0, q_dtype=kind)[1])
        assert not z.any()


@pytest.mark.parametrize("kind", [0, 1])
def test_norm_float32_rows_of_any_magnitude(g, kind):  # noqa: F811
    """Rows whose squares leave float32 on either side, beside ordinary ones."""
    rng = np.random.default_rng(2)
    # magnitude of a row; with normal values and weights below 2, products stay finite and normal
    mags = np.array([1, 1e-34, 1e-28, 1e-22, 1e-19, 1e-15, 1e-7, 1e15, 1e18, 1e19, 1e20, 1e28, 1e36])
    for K in WIDTHS:
        base = rng.standard_normal((len(mags), K))
        base[:, 0] = 1
        x = (np.clip(base, -5, 5) * mags[:, None]).astype(np.float32)
        w = (1 + 0.2 * np.clip(rng.standard_normal(K), -4, 4)).astype(np.float32)
        r = (0.5 * x[:, ::-1]).copy()
        for eps in (0.0, 1e-44, 1e-36, 1e-5, 1e30):
            for res in (None, r):
                say("magnitudes", K, eps, kind, res is not None)
                codes, scale, _ = (host(t) for t in g.add_rmsnorm_q8(
                    dev(x), dev(w), None if res is None else dev(res), eps=eps, q_dtype=kind))
                assert np.isfinite(scale).all()
                check_norm(codes, scale, x, w, res, eps, kind, (K, eps, kind))


def test_norm_float32_row_at_the_largest_values(g):  # noqa: F811
    """Weights that bring the largest rows down and the smallest up."""
    rng = np.random.default_rng(3)
    for K in WIDTHS:
        s = np.sign(rng.standard_normal((1, K)))
        for h, w, eps in ((3e38, 1e-6, 0.0), (3e38, 1e-30, 1e-5), (1e-37, 100.0, 0.0), (1e-30, 1e20, 0.0)):
            x = (h * s).astype(np.float32)
            W = np.full(K, w, np.float32)
            codes, scale, _ = (host(t) for t in g.add_rmsnorm_q8(dev(x), dev(W), eps=eps))
            check_norm(codes, scale, x, W, None, eps, 0, (K, h, w, eps))


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("D,rot,style,n,page", [(64, 0, 0, 1, 16), (100, 100, 0, 5, 16), (128, 64, 1, 9, 16),
                                                (128, 128, 0, 100, 128), (100, 100, 0, 120, 128)])
def test_append_continues_pages_of_any_scale(g, D, rot, style, n, page, kind):  # noqa: F811
    """Pages filled by someone else: their scales are no powers of two, some subnormal;
    new elements that are ties of the codes in units of them, and zeros."""
    rng = np.random.default_rng(D)
    Hkv, B, lead = 2, 24, 5
    dp = g.kv8_padded_dim(D)
    cache = O.PagedCache8(B, page, Hkv, D, dp, kind)
    for c in cache.codes:
        c[:, :, :lead, :D] = rng.integers(0, 0x70, (B, Hkv, lead, D))
    for s in cache.scale:
        s[:] = np.exp(rng.uniform(-8, 3, s.shape)).astype(np.float32)
        s[3], s[4], s[5], s[B - 2], s[B - 1] = 1e-40, 2.0 ** -127, 3e-38, 2.0 ** 127, 1.5 * 2.0 ** 126
    table = np.arange(B, dtype=np.int32)[rng.permutation(B), None]
    cdev = (device_codes(cache, 0), device_codes(cache, 1), dev(cache.scale[0]), dev(cache.scale[1]))
    tab = rope_table(page, rot) if rot else None
    if rot:
        tab[:, :rot // 2], tab[:, rot // 2:] = 1, 0          # the turn keeps the ties
    new = []
    for s in cache.scale:
        if kind == 0:
            t = rng.integers(-100, 100, (B, n, Hkv, D)) + 0.5
        else:
            t = (rng.integers(8, 16, (B, n, Hkv, D)) + 0.5) * 2.0 ** rng.integers(-6, 4, (B, n, Hkv, D))
        t[table[:, 0] >= B - 2] /= 1024                       # products that stay finite
        x = (t * s[table[:, 0]][:, None, :, None]).astype(np.float32)
        x[rng.random(x.shape) < 0.1] = 0
        x[table[:, 0] == 3] = x[table[:, 0] == 4] = 0
        new.append(x.reshape(B * n, Hkv, D))
    append_call(g, cdev, (new[0], *new), table, [lead + n] * B, [n] * B, tab, style, np.float32, False,
                with_q=False)
    pos = np.tile(np.arange(lead, lead + n), B)
    kr = O.rope_f32(new[0], tab, pos, rot, style)
    for b in range(B):
        cache.append((kr[b * n:(b + 1) * n], new[1][b * n:(b + 1) * n]), table[b], lead)
    check_cache(cache, *cdev, (D, kind))


def long_and_singles(batch, n, page):
    """One sequence of n new tokens at the front of a batch of single ones: lengths,
    q_indptr, page table and pool."""
    news = np.array([n] + [1] * (batch - 1))
    lens = news + np.arange(batch) % page
    need = -(-lens // page)
    table = np.full((batch, need.max()), -1, np.int32)
    first = np.concatenate([[0], np.cumsum(need)])
    for b in range(batch):
        table[b, :need[b]] = first[b] + np.arange(need[b])
    return lens.astype(np.int32), np.concatenate([[0], np.cumsum(news)]).astype(np.int32), table, int(first[-1])


def test_append_of_a_long_prompt_in_a_large_batch(g):  # noqa: F811
    """More blocks than one grid dimension launches: the same as the long sequence and
    the others in calls of their own."""
    batch, n, page, H, D = 1024, 16384, 16, 8, 64
    lens, indptr, table, pool = long_and_singles(batch, n, page)
    T = int(indptr[-1])
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(T, H, D, device="cuda", generator=gen).half() for _ in range(3))
    rope = dev(rope_table(n + page, D))
    out = []
    for calls in ([(0, batch, n)], [(0, 1, n), (1, batch, 1)]):
        c = g.kv8_alloc(pool, page, H, D)
        qo = []
        for a, z, most in calls:
            rows = slice(int(indptr[a]), int(indptr[z]))
            say("append", a, z, "rows", rows)
            qo.append(g.rope_append_kv8(q[rows], k[rows], v[rows], *c, dev(table[a:z]), dev(lens[a:z]),
                                        q_indptr=dev(indptr[a:z + 1] - indptr[a]), max_q=most, rope=rope))
        out.append((*c, torch.cat(qo)))
    torch.cuda.synchronize()
    for a, b in zip(*out):
        assert torch.equal(a, b)
    assert all(bool(t.any()) for t in out[0])


def test_attention_of_a_long_prompt_in_a_large_batch(g):  # noqa: F811
    """The same for attention: sampled rows against the oracle."""
    batch, n, page, H, D = 4096, 12400, 64, 32, 4
    lens, indptr, table, pool = long_and_singles(batch, n, page)
    T = int(indptr[-1])
    gen = torch.Generator(device="cuda").manual_seed(2)
    c = (torch.randint(-127, 128, (pool, H, page, 64), device="cuda", generator=gen).to(torch.int8),
         torch.randint(-127, 128, (pool, H, 64, page), device="cuda", generator=gen).to(torch.int8),
         *(torch.rand(pool, H, device="cuda", generator=gen) / 40 for _ in range(2)))
    c[0][..., D:] = 0
    c[1][:, :, D:] = 0
    q = torch.randn(T, H, D, device="cuda", generator=gen).half()
    say("attention", batch, T)
    out = host(g.paged_attn_kv8(q, *c, dev(table), dev(lens), int(lens.max()), q_indptr=dev(indptr),
                                max_q=T)).astype(np.float64)
    assert np.isfinite(out).all()
    qh = host(q)
    for b, i in [(0, 0), (0, 255), (0, 6001), (0, n - 1), (1, 0), (77, 0), (batch - 1, 0)]:
        ids = torch.from_numpy(table[b, :-(-int(lens[b]) // page)].astype(np.int64)).cuda()
        for h in (0, 31):
            k = host(c[0][ids, h, :, :D].double() * c[2][ids, h].double()[:, None, None]).reshape(-1, D)
            v = host((c[1][ids, h, :D].double() * c[3][ids, h].double()[:, None, None]).transpose(1, 2)
                     .contiguous()).reshape(-1, D)
            row, new = int(indptr[b]) + i, int(indptr[b + 1] - indptr[b])
            ref, _, absv, terms = O.attention_rows(qh[row:row + 1, h], k, v, [int(lens[b]) - new + i + 1],
                                                   D ** -0.5)
            assert np.all(np.abs(out[row:row + 1, h] - ref) <= attn_bound(ref, absv, terms, int(lens[b]), D)), \
                (b, i, h)


@pytest.mark.parametrize("given", [False, True])
def test_append_of_more_sequences_than_a_grid_has_rows(g, given):  # noqa: F811
    """70000 single tokens, with and without q_indptr: the same as in two calls."""
    batch, half, H, D, page = 70000, 35000, 1, 64, 16
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(batch, H, D, device="cuda", generator=gen).half() for _ in range(3))
    lens = dev((1 + np.arange(batch) % page).astype(np.int32))
    table = dev(np.arange(batch, dtype=np.int32)[:, None])
    rope = dev(rope_table(page, D))
    out = []
    for calls in ([(0, batch)], [(0, half), (half, batch)]):
        c = g.kv8_alloc(batch, page, H, D)
        qo = []
        for a, z in calls:
            ip = dev(np.arange(z - a + 1, dtype=np.int32)) if given else None
            say("append", a, z, given)
            qo.append(g.rope_append_kv8(q[a:z], k[a:z], v[a:z], *c, table[a:z], lens[a:z], q_indptr=ip,
                                        rope=rope))
        out.append((*c, torch.cat(qo)))
    torch.cuda.synchronize()
    for a, b in zip(*out):
        assert torch.equal(a, b)
    assert bool((out[0][2] > 0).all())
