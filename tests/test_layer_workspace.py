"""Host-only: the places where split attention keeps its partial results lie inside
the workspace that the call asks for, and no two sequences share one. The library
numbers them here with the function that its kernels use."""
import ctypes

import numpy as np
import pytest

import gemv_nibble_unpack_amd as G

COUNTERS = 16384        # arrival counters at the start of a workspace


def part_slots(news, max_q, max_kv, Hq, Hkv, D, indptr=None, tokens=None):
    """(reported bytes, slots in use, bytes of one) of a split call, None if it is not."""
    fn = G.load().w4_attn_part_slots
    fn.restype = ctypes.c_int64
    fn.argtypes = [ctypes.c_int] * 7 + [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.POINTER(ctypes.c_int64)]
    if indptr is None:
        indptr = np.concatenate([[0], np.cumsum(news)])
    indptr = np.asarray(indptr, np.int32)
    tokens = int(indptr[-1]) if tokens is None else tokens
    sizes = (len(indptr) - 1, tokens, max_q, max_kv, Hq, Hkv, D)
    need = G.paged_attn_kv8_workspace_bytes(*sizes)
    slots, each = np.full(1 << 16, -1, np.int64), ctypes.c_int64()
    n = fn(*sizes, indptr.ctypes.data, slots.ctypes.data, slots.size, ctypes.byref(each))
    assert n <= slots.size
    return None if n == 0 else (need, slots[:n][slots[:n] >= 0], each.value)


def check(*a, **kw):
    """True if the call is split; its parts must fit."""
    r = part_slots(*a, **kw)
    if r is None:
        return False
    need, slots, each = r
    assert need <= G.W4_ATTN_WORKSPACE_MAX, (a, kw)
    assert COUNTERS + (int(slots.max(initial=-1)) + 1) * each <= need, (a, kw)
    return True


def distinct(*a, **kw):
    r = part_slots(*a, **kw)
    assert r is None or len(np.unique(r[1])) == len(r[1]), (a, kw)


@pytest.mark.parametrize("batch,new,kv,Hq,Hkv,D", [
    (2, 64, 4096, 32, 8, 128), (4, 64, 4096, 32, 8, 128), (16, 17, 4096, 32, 8, 128),
    (8, 64, 4096, 32, 8, 128), (8, 64, 16384, 32, 8, 128), (20, 64, 16384, 32, 8, 128),
    (2, 128, 8192, 32, 8, 128), (2, 128, 16384, 16, 16, 256), (3, 65, 9000, 1, 1, 192)])
def test_equal_chunks_fit(batch, new, kv, Hq, Hkv, D):
    assert check([new] * batch, new, kv, Hq, Hkv, D)
    distinct([new] * batch, new, kv, Hq, Hkv, D)


def test_random_batches_fit():
    rng = np.random.default_rng(0)
    split = 0
    for i in range(4000):
        batch = int(rng.integers(1, 40))
        Hkv = int(rng.choice([1, 2, 7, 8, 16]))
        Hq = Hkv * int(rng.choice([1, 2, 4, 5, 8]))
        D = int(rng.choice([64, 96, 100, 128, 192, 256]))
        most = int(np.exp(rng.uniform(0, 8)))
        kind = i % 4
        if kind == 0:                        # equal
            news = [most] * batch
        elif kind == 1:                      # similar
            news = (most + rng.integers(0, 3, batch)).tolist()
        elif kind == 2:                      # ragged, empty ones among them
            news = rng.integers(0, most + 1, batch).tolist()
        else:                                # one long
            news = [1] * batch
            news[int(rng.integers(batch))] = most
        if sum(news) == 0:
            continue
        # a bound on the new tokens that is exact, loose or (some rows left out) low
        max_q = max(1, int(max(news) * rng.choice([1, 1, 1, 2, 0.4])))
        args = (news, max_q, int(np.exp(rng.uniform(3, 12))), Hq, Hkv, D)
        split += check(*args)
        distinct(*args)
    assert split > 1500


def test_one_tile_exactly_filled_fits():
    for D, rows in ((128, 256), (256, 128)):
        for group in (1, 4, 8):
            for batch in (1, 2, 3, 9):
                for more in (-1, 0, 1):
                    n = rows // group + more
                    args = ([n] * batch, n, 20000, group, 1, D)
                    check(*args)
                    distinct(*args)


def test_lengths_that_contradict_the_bound_fit():
    """Rows before the first sequence, and more new tokens than max_q."""
    for D in (64, 128, 256):
        for max_q in (70, 128, 300):
            assert check(None, max_q, 30000, 4, 1, D, indptr=[900, 1000])
            assert check(None, max_q, 30000, 4, 1, D, indptr=[0, 990, 1000])
            assert check(None, max_q, 30000, 4, 1, D, indptr=[500, 500, 400, 1000, 70], tokens=1000)


@pytest.mark.parametrize("max_q", [1, 5, 200])
def test_nothing_cached_needs_no_workspace(max_q):
    """A bound of zero on the cached tokens is a size like others."""
    for batch in (1, 3, 100):
        for D in (64, 256):
            assert G.paged_attn_kv8_workspace_bytes(batch, batch * max_q, max_q, 0, 8, 2, D) == 0
