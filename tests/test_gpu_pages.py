"""GPU parity of the page bookkeeping and the writes into pages: whole numbers
and copies, so everything is compared bit for bit with the oracle."""
import numpy as np
import pytest
import torch

from gpu_util import dev, host, zeros_status
from oracle import paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dflv():
    import speculative_decoding_tree_layer_gb300 as pkg

    pkg.build()
    pkg.load()
    return pkg


def pool(rng, past, width, page, spare):
    """Tables that hold exactly the committed tokens' pages, and the free list."""
    B = len(past)
    held = -(-past // page)
    n_pages = int(held.sum()) + spare
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    used = 0
    for b in range(B):
        table[b, :held[b]] = ids[used:used + held[b]]
        used += held[b]
    free = np.full(n_pages, -1, np.int32)
    free[:n_pages - used] = ids[used:]
    return table, held.astype(np.int32), free, n_pages - used


def grow(dflv, past, new, held, free, n_free, table, page, N):
    d = dict(past=dev(past), new=dev(new), held=dev(held), free=dev(free),
             n_free=dev(np.array([n_free], np.int32)), table=dev(table),
             slots=torch.full((len(past), N), -7, dtype=torch.int32, device="cuda"), st=zeros_status())
    desc = dflv.pages_desc(len(past), N, page, len(free), table.shape[1])
    dflv.check(dflv.dflv_block_tables_grow(desc, d["past"], d["new"], d["held"], d["free"], d["n_free"], d["table"],
                                           d["slots"], d["st"]))
    return desc, d


SHAPES = [(1, 1, 16, 0), (1, 1, 16, 16), (8, 22, 16, 300), (257, 5, 32, 40), (3, 64, 128, 1000), (600, 7, 64, 90),
          (2, 9001, 16, 33), (40, 4096, 16, 0), (1, 100003, 128, 5)]


@pytest.mark.parametrize("B,N,page,past_max", SHAPES)
def test_grow_and_release(dflv, B, N, page, past_max):
    rng = np.random.default_rng(B * N + page)
    past = rng.integers(0, past_max + 1, B).astype(np.int32)
    new = rng.integers(0, N + 1, B).astype(np.int32)
    new[-1] = N
    width = -(-(past_max + N) // page) + 1
    table, held, free, n_free = pool(rng, past, width, page, int((-(-new // page) + 1).sum()))
    rh, rf, rt, rs, st = paged.tables_grow(past, new, held, free, n_free, table, page, N)
    assert st == 0
    desc, d = grow(dflv, past, new, held, free, n_free, table, page, N)
    assert int(d["st"]) == 0
    for name, ref in (("table", rt), ("slots", rs), ("held", rh), ("n_free", [rf]), ("free", free)):
        assert np.array_equal(host(d[name]), ref), name
    # the step's tokens but a few go back
    keep = (past + rng.integers(0, 2, B) * (new // 2)).astype(np.int32)
    rh2, rfree, rf2, st = paged.tables_release(keep, rh, free, rf, rt, page)
    dflv.check(dflv.dflv_block_tables_release(desc, dev(keep), d["held"], d["free"], d["n_free"], d["table"], d["st"]))
    assert st == 0 and int(d["st"]) == 0
    for name, ref in (("table", rt), ("held", rh2), ("n_free", [rf2]), ("free", rfree)):
        assert np.array_equal(host(d[name]), ref), name
    # and the rest: the sequences end
    dflv.check(dflv.dflv_block_tables_release(desc, dev(np.zeros(B, np.int32)), d["held"], d["free"], d["n_free"],
                                              d["table"], d["st"]))
    assert int(d["n_free"]) == len(free) and not host(d["held"]).any()
    assert sorted(host(d["free"]).tolist()) == list(range(len(free)))


@pytest.mark.parametrize("B", [5, 700])
def test_grow_when_pages_run_out(dflv, B):
    rng = np.random.default_rng(B)
    page, N, width = 16, 40, 6
    past = rng.integers(0, 40, B).astype(np.int32)
    new = rng.integers(0, N + 1, B).astype(np.int32)
    need = -(-(past + new) // page) - -(-past // page)
    table, held, free, n_free = pool(rng, past, width, page, int(need.sum() * 0.6))
    rh, rf, rt, rs, st = paged.tables_grow(past, new, held, free, n_free, table, page, N)
    assert st == paged.DEV_CAPACITY
    _, d = grow(dflv, past, new, held, free, n_free, table, page, N)
    assert int(d["st"]) == st
    for name, ref in (("table", rt), ("slots", rs), ("held", rh), ("n_free", [rf])):
        assert np.array_equal(host(d[name]), ref), name


def test_lengths_out_of_range(dflv):
    page, N, width, B = 16, 20, 4, 6
    past = np.array([0, -1, 60, 3, 5, 1 << 30], np.int32)
    new = np.array([5, 5, 20, 21, -2, 4], np.int32)
    held = np.array([0, 0, 4, 1, 9, 4], np.int32)
    table = np.arange(B * width, dtype=np.int32).reshape(B, width)
    free = np.arange(100, 164, dtype=np.int32) % 64
    rh, rf, rt, rs, st = paged.tables_grow(past, new, held, free, 40, table, page, N)
    _, d = grow(dflv, past, new, held, free, 40, table, page, N)
    assert int(d["st"]) == st == paged.DEV_CAPACITY
    for name, ref in (("table", rt), ("slots", rs), ("held", rh), ("n_free", [rf])):
        assert np.array_equal(host(d[name]), ref), name


def test_release_refuses_what_does_not_fit(dflv):
    page, width, B = 16, 4, 3
    desc = dflv.pages_desc(B, 1, page, 8, width)
    table = np.array([[0, 1, 2, 3], [4, 5, 9, -1], [6, 7, 0, 0]], np.int32)

    def call(keep, held, n_free):
        t = [dev(np.array(x, np.int32)) for x in (keep, held, [n_free])]
        free, st = torch.full((8,), -1, dtype=torch.int32, device="cuda"), zeros_status()
        dflv.check(dflv.dflv_block_tables_release(desc, t[0], t[1], free, t[2], dev(table), st))
        ref = paged.tables_release(np.array(keep), np.array(held, np.int32), np.full(8, -1, np.int32), n_free, table,
                                   page)
        assert int(st) == ref[3]
        assert np.array_equal(host(t[1]), ref[0]) and int(t[2]) == ref[2] and np.array_equal(host(free), ref[1])
        return int(st)

    assert call([16, 0, 0], [2, 2, 1], 0) == 0
    assert call([-1, 0, 0], [2, 2, 1], 0) == paged.DEV_CAPACITY      # negative length
    assert call([33, 0, 0], [2, 2, 1], 0) == paged.DEV_CAPACITY      # keeps more than it holds
    assert call([0, 0, 0], [5, 2, 1], 0) == paged.DEV_CAPACITY       # holds more than the row
    assert call([0, 0, 0], [2, 2, 1], 4) == paged.DEV_CAPACITY       # no room: nothing happens
    assert call([0, 0, 0], [2, 3, 1], 0) == paged.DEV_PAGE           # page 9 of 8


def planes(rng, n_pages, Hkv, page, D):
    return [rng.integers(0, 1 << 16, (n_pages, Hkv, page, D)).astype(np.uint16) for _ in range(2)]


@pytest.mark.parametrize("B,N,Hkv,D,page", [(1, 1, 1, 64, 16), (3, 7, 2, 64, 32), (2, 300, 4, 128, 16),
                                            (5, 64, 3, 256, 64), (64, 1, 8, 128, 128)])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_append(dflv, B, N, Hkv, D, page, kind):
    rng = np.random.default_rng(B * N + D)
    n_pages = -(-B * N // page) + 3
    k, v = planes(rng, n_pages, Hkv, page, D)
    slots = rng.permutation(n_pages * page)[:B * N].reshape(B, N).astype(np.int32)
    slots[rng.random((B, N)) < 0.2] = -1
    kn, vn = (rng.integers(0, 1 << 16, (B, N, Hkv, D)).astype(np.uint16) for _ in range(2))
    t = torch.bfloat16 if kind == "bf16" else torch.float16
    dk, dv, dkn, dvn = (dev(x).view(t) for x in (k, v, kn, vn))
    st = zeros_status()
    desc = dflv.paged_kv_desc(B, N, Hkv, D, page, n_pages, dflv.DFLV_KV_BF16 if kind == "bf16" else dflv.DFLV_KV_F16)
    dflv.check(dflv.dflv_paged_kv_append(desc, dev(slots), dkn, dvn, dflv.kv_layer(dk, dv), st))
    paged.paged_append(slots, kn, vn, k, v)
    assert int(st) == 0
    assert np.array_equal(host(dk.view(torch.int16)).view(np.uint16), k)
    assert np.array_equal(host(dv.view(torch.int16)).view(np.uint16), v)


def test_append_from_a_fused_projection_and_bad_slots(dflv):
    rng = np.random.default_rng(9)
    B, N, Hkv, D, page, n_pages = 2, 5, 2, 64, 16, 4
    k, v = planes(rng, n_pages, Hkv, page, D)
    slots = np.array([[3, 17, -1, 64, 20], [-5, 63, 0, 1 << 30, 31]], np.int32)
    wide = torch.randn(B, N, 3 * Hkv * D, device="cuda").bfloat16()
    kn, vn = (wide[:, :, o * Hkv * D:(o + 1) * Hkv * D].unflatten(2, (Hkv, D)) for o in (1, 2))
    dk, dv, st = dev(k), dev(v), zeros_status()
    desc = dflv.paged_kv_desc(B, N, Hkv, D, page, n_pages, dflv.DFLV_KV_BF16, 3 * Hkv * D)
    dflv.check(dflv.dflv_paged_kv_append(desc, dev(slots), kn, vn, dflv.kv_layer(dk, dv), st))
    bits = lambda x: host(x.contiguous().view(torch.int16)).view(np.uint16)  # noqa: E731
    paged.paged_append(slots, bits(kn), bits(vn), k, v)
    assert int(st) == paged.DEV_PAGE
    assert np.array_equal(host(dk).view(np.uint16), k) and np.array_equal(host(dv).view(np.uint16), v)
    # the same view without its stride, or with another one, is refused
    for stride in (0, 4 * Hkv * D):
        desc = dflv.paged_kv_desc(B, N, Hkv, D, page, n_pages, dflv.DFLV_KV_BF16, stride)
        assert dflv.dflv_paged_kv_append(desc, dev(slots), kn, vn, dflv.kv_layer(dk, dv),
                                         st) == dflv.DFLV_ERR_INVALID_ARG


@pytest.mark.parametrize("B,N,Hkv,D,page,layers", [(1, 1, 1, 64, 16, 1), (4, 22, 4, 256, 16, 3), (3, 64, 2, 64, 32, 2),
                                                   (2, 64, 1, 128, 128, 64)])
def test_commit(dflv, B, N, Hkv, D, page, layers):
    rng = np.random.default_rng(N + D + layers)
    n_pages = -(-B * N // page) + 2
    ks, vs = zip(*[planes(rng, n_pages, Hkv, page, D) for _ in range(layers)])
    slots = rng.permutation(n_pages * page)[:B * N].reshape(B, N).astype(np.int32)
    path = np.full((B, N), 1 << 20, np.int32)
    plen = np.zeros(B, np.int32)
    for b in range(B):
        # all of the nodes, every second one, none, the first
        p = [list(range(N)), list(range(0, N, 2)), [], [0]][b % 4]
        path[b, :len(p)], plen[b] = p, len(p)
    past = rng.integers(0, 1000, B).astype(np.int32)
    dk, dv, dp, st = [dev(x) for x in ks], [dev(x) for x in vs], dev(past), zeros_status()
    desc = dflv.paged_kv_desc(B, N, Hkv, D, page, n_pages, dflv.DFLV_KV_F16)
    caches = [dflv.kv_layer(a, b) for a, b in zip(dk, dv)]
    dflv.check(dflv.dflv_paged_kv_commit(desc, layers, caches, dev(slots), dev(path), dev(plen), dp, st))
    paged.paged_commit(slots, path, plen, list(ks) + list(vs))
    assert int(st) == 0 and np.array_equal(host(dp), past + plen)
    for got, ref in zip(dk + dv, list(ks) + list(vs)):
        assert np.array_equal(host(got).view(np.uint16), ref)


@pytest.mark.parametrize("path,plen,slot,bits", [
    ([0, 2, 1], 3, 5, paged.DEV_PATH), ([0, 1, 1], 3, 5, paged.DEV_PATH), ([0, 4, 0], 2, 5, paged.DEV_PATH),
    ([0, -1, 0], 2, 5, paged.DEV_PATH), ([0, 1, 2], 5, 5, paged.DEV_PATH), ([0, 1, 2], -1, 5, paged.DEV_PATH),
    ([0, 2, 3], 3, -1, paged.DEV_PAGE), ([0, 2, 3], 3, 64, paged.DEV_PAGE)])
def test_commit_leaves_a_bad_sequence_alone(dflv, path, plen, slot, bits):
    rng = np.random.default_rng(3)
    N, Hkv, D, page, n_pages = 4, 2, 64, 16, 4
    k, v = planes(rng, n_pages, Hkv, page, D)
    slots = np.array([[10, 11, slot, 13]], np.int32)
    dk, dv, past, st = dev(k), dev(v), dev(np.array([7], np.int32)), zeros_status()
    desc = dflv.paged_kv_desc(1, N, Hkv, D, page, n_pages, dflv.DFLV_KV_BF16)
    dflv.check(dflv.dflv_paged_kv_commit(desc, 1, [dflv.kv_layer(dk, dv)], dev(slots),
                                         dev(np.array([path + [0]], np.int32)), dev(np.array([plen], np.int32)), past,
                                         st))
    assert int(st) == bits and int(past) == 7
    assert np.array_equal(host(dk).view(np.uint16), k) and np.array_equal(host(dv).view(np.uint16), v)


@pytest.mark.parametrize("B,N", [(3, 40), (3, 41), (300, 44), (300, 33)])
@pytest.mark.parametrize("bad", [-1, -(1 << 31), 0, 3, 1 << 27, (1 << 28) + 1, (1 << 31) - 1])
def test_grow_gives_no_slots_in_pages_outside_the_pool(dflv, B, N, bad):
    # damaged ids in held pages and in the free list, some of which name a page of
    # the pool once they are shifted to a slot (ids 0 and 3 stand for one past it)
    rng = np.random.default_rng(B + N)
    page, width = 16, 8
    past = rng.integers(1, 40, B).astype(np.int32)
    new = rng.integers(1, N + 1, B).astype(np.int32)
    table, held, free, n_free = pool(rng, past, width, page, int((-(-new // page) + 1).sum()))
    bad = len(free) + bad if bad in (0, 3) else bad
    for b in range(0, B, 3):
        table[b, held[b] - 1] = bad
    free[n_free - 1 - rng.integers(0, n_free // 2, max(1, B // 8))] = bad
    rh, rf, rt, rs, st = paged.tables_grow(past, new, held, free, n_free, table, page, N)
    assert st == paged.DEV_PAGE
    _, d = grow(dflv, past, new, held, free, n_free, table, page, N)
    assert int(d["st"]) == st
    for name, ref in (("table", rt), ("slots", rs), ("held", rh), ("n_free", [rf]), ("free", free)):
        assert np.array_equal(host(d[name]), ref), name
    # a damaged page that no new token lies in is not looked at
    table[:, 0] = bad
    past = (held * page).astype(np.int32)
    free[:n_free] = np.arange(n_free)
    rh, rf, rt, rs, st = paged.tables_grow(past, new, held, free, n_free, table, page, N)
    _, d = grow(dflv, past, new, held, free, n_free, table, page, N)
    assert st == 0 and int(d["st"]) == 0 and np.array_equal(host(d["slots"]), rs)


def test_as_many_sequences_as_there_may_be(dflv):
    # 2^20 of them: three in four need a page, and the last ones get none
    B, page = 1 << 20, 16
    rng = np.random.default_rng(6)
    new = (rng.random(B) < 0.75).astype(np.int32)
    n_free = int(new.sum()) - 1000
    free = rng.permutation(n_free + 5).astype(np.int32)
    zero, table = np.zeros(B, np.int32), np.full((B, 1), -1, np.int32)
    desc, d = grow(dflv, zero, new, zero, free, n_free, table, page, 1)
    rank = np.cumsum(new) - new
    served = (new > 0) & (rank < n_free)
    ids = np.where(served, free[np.clip(n_free - 1 - rank, 0, None)], -1)
    assert int(d["st"]) == dflv.DFLV_DEV_CAPACITY and int(d["n_free"]) == 0
    assert np.array_equal(host(d["held"]), served) and np.array_equal(host(d["table"])[:, 0], ids)
    assert np.array_equal(host(d["slots"])[:, 0], np.where(served, ids * page, -1))
    d["st"].zero_()
    dflv.check(dflv.dflv_block_tables_release(desc, dev(zero), d["held"], d["free"], d["n_free"], d["table"], d["st"]))
    assert int(d["st"]) == 0 and int(d["n_free"]) == n_free and not host(d["held"]).any()
    assert np.array_equal(host(d["free"]), free)
