"""GPU: split attention stays inside a workspace of exactly the size that it asks for
(the bytes behind it keep their pattern), at the batches whose parts are numbered
by row tile and by row, against a float64 reference."""
import numpy as np
import pytest

from tests._helpers import say
from tests.test_gpu_layer import attn_bound, dev, device_codes, g, host, random_cache  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

GUARD = 1 << 20


def exact_workspace(g, batch, tokens, max_q, max_kv, Hq, Hkv, D):
    """A buffer whose first bytes are the workspace, and what lies behind it."""
    need = g.paged_attn_kv8_workspace_bytes(batch, tokens, max_q, max_kv, Hq, Hkv, D)
    assert need > 0, "this call is not split"
    # room for twice the size: parts past the end would land in the buffer
    buf = torch.full((2 * need + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    buf[:need].zero_()
    return buf, need


def check_split(g, rng, lens, indptr, max_q, Hq, Hkv, D, page, kind, max_kv=None):
    max_kv = max(lens) if max_kv is None else max_kv
    cache, table = random_cache(rng, lens, page, Hkv, D, g.kv8_padded_dim(D), kind)
    T, G = int(indptr[-1]), Hq // Hkv
    q = rng.standard_normal((T, Hq, D)).astype(np.float16)
    buf, need = exact_workspace(g, len(lens), T, max_q, max_kv, Hq, Hkv, D)
    keep = torch.full((T, Hq, D), 5.0, dtype=torch.float16, device="cuda")
    args = (dev(q), device_codes(cache, 0), device_codes(cache, 1), dev(cache.scale[0]),
            dev(cache.scale[1]), dev(table), dev(np.asarray(lens, np.int32)), max_kv)
    kw = dict(q_indptr=dev(np.asarray(indptr, np.int32)), max_q=max_q, workspace=buf[:need], out=keep)
    say("split", lens[:4], list(indptr[:4]), Hq, Hkv, D, "workspace", need)
    got = host(g.paged_attn_kv8(*args, **kw)).astype(np.float64)
    assert bool((buf[need:] == 0xA5).all()), "written behind the workspace"
    assert not buf[:16384].any()                 # arrival counters left zero
    again = host(g.paged_attn_kv8(*args, **kw)).astype(np.float64)
    assert np.array_equal(again, got, equal_nan=True)
    rows_done = np.zeros(T, bool)
    for b, n in enumerate(np.diff(indptr)):
        row = int(indptr[b])
        rows_done[row:row + n] = True
        if n > max_q:
            assert np.isnan(got[row:row + max_q]).all() and (got[row + max_q:row + n] == 5.0).all()
            continue
        for h in range(Hkv if n else 0):
            k, v = (cache.rows(w, table[b], lens[b], h) for w in range(2))
            qs = q[row:row + n, h * G:(h + 1) * G].reshape(n * G, D).astype(np.float64)
            limit = np.repeat(lens[b] - n + 1 + np.arange(n), G)
            s = qs @ k.T * D ** -0.5
            s[np.arange(lens[b])[None] >= limit[:, None]] = -np.inf
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            terms = (np.abs(qs) @ np.abs(k).T).max(1) * D ** -0.5
            o = got[row:row + n, h * G:(h + 1) * G].reshape(n * G, D)
            err = np.abs(o - w @ v) - attn_bound(w @ v, w @ np.abs(v), terms, lens[b], D)
            assert np.all(err <= 0), (b, h, float(err.max()))
    assert (got[~rows_done] == 5.0).all()


@pytest.mark.parametrize("batch,new,kv,Hq,Hkv,D,kind", [
    (2, 64, 4096, 32, 8, 128, 0), (8, 64, 4096, 32, 8, 128, 1), (3, 65, 3000, 4, 2, 64, 0),
    (2, 128, 5000, 4, 4, 256, 1), (4, 17, 4096, 32, 8, 128, 0), (3, 43, 2600, 6, 2, 192, 0)])
def test_equal_chunks_stay_inside(g, batch, new, kv, Hq, Hkv, D, kind):  # noqa: F811
    rng = np.random.default_rng(batch + new)
    check_split(g, rng, [kv] * batch, np.arange(batch + 1) * new, new, Hq, Hkv, D, 64, kind)


@pytest.mark.parametrize("D", [64, 256])
def test_ragged_chunks_stay_inside(g, D):  # noqa: F811
    rng = np.random.default_rng(D)
    news = [300, 1, 0, 70, 300, 2, 5, 1]
    lens = [4000, 900, 30, 2500, 300, 1000, 5, 1]
    check_split(g, rng, lens, np.concatenate([[0], np.cumsum(news)]), 300, 4, 2, D, 32, 0)


@pytest.mark.parametrize("D", [128, 192])
def test_rows_before_the_first_and_past_max_q_stay_inside(g, D):  # noqa: F811
    rng = np.random.default_rng(D + 1)
    check_split(g, rng, [5000], [900, 1000], 100, 4, 1, D, 64, 1)
    check_split(g, rng, [5000, 3000], [0, 400, 500], 100, 4, 1, D, 64, 0)


@pytest.mark.parametrize("n", [1, 5, 200])
def test_nothing_cached(g, n):  # noqa: F811
    """max_kv = 0: every row sees nothing; a longer sequence does not fit the bound."""
    rng = np.random.default_rng(n)
    cache, table = random_cache(rng, [20, 20], 16, 1, 64, 64, 0)
    cd = (device_codes(cache, 0), device_codes(cache, 1), dev(cache.scale[0]), dev(cache.scale[1]),
          dev(table))
    q = dev(rng.standard_normal((2 * n, 2, 64)).astype(np.float16))
    indptr = dev(np.array([0, n, 2 * n], np.int32))
    lse = torch.zeros(2 * n, 2, device="cuda")
    for lens in ([0, 0], [0, 20]):
        out = host(g.paged_attn_kv8(q, *cd, dev(np.array(lens, np.int32)), 0, q_indptr=indptr, max_q=n,
                                    lse=lse))
        assert not out[:n].any() and np.isneginf(host(lse)[:n]).all()
        if lens[1]:
            assert np.isnan(out[n:]).all() and np.isnan(host(lse)[n:]).all()
        else:
            assert not out[n:].any() and np.isneginf(host(lse)[n:]).all()
