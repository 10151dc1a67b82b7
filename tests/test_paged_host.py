"""Host-side checks of the paged-cache, shared-prefix and sampling calls: what
they refuse before anything is launched (CPU only: no call here reaches a
kernel), and the oracle's own pins."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_tree_layer_gb300 as pkg
from oracle import paged
from speculative_decoding_tree_layer_gb300 import dflv

P = 16  # a well-aligned address that nothing reads
BAD, UNS, CAP = dflv.DFLV_ERR_INVALID_ARG, dflv.DFLV_ERR_UNSUPPORTED, dflv.DFLV_ERR_CAPACITY


@pytest.fixture(scope="module", autouse=True)
def lib():
    pkg.build()
    return dflv.load()


def grow(d, **over):
    a = dict(n_past=P, n_new=P, n_held=P, free_list=P, n_free=P, table=P, slots=P, status_dev=P)
    a.update(over)
    return dflv.dflv_block_tables_grow(d, stream=0, **a)


def release(d, **over):
    a = dict(keep_len=P, n_held=P, free_list=P, n_free=P, table=P, status_dev=P)
    a.update(over)
    return dflv.dflv_block_tables_release(d, stream=0, **a)


@pytest.mark.parametrize("call", [grow, release])
@pytest.mark.parametrize("shape,code", [
    ((0, 1, 16, 8, 8), BAD), ((1, 0, 16, 8, 8), BAD), ((1, 1, 16, 0, 8), BAD), ((1, 1, 16, 8, 0), BAD),
    ((1, 1, 0, 8, 8), BAD), ((1, 1, 16, 8, 8, 1), BAD),
    ((1, 1, 8, 8, 8), UNS), ((1, 1, 48, 8, 8), UNS), ((1, 1, 256, 8, 8), UNS),
    ((1 << 16, 1 << 15, 16, 8, 8), UNS), ((1 << 16, 1, 16, 8, 1 << 15), UNS), ((1, 1, 128, 1 << 24, 8), UNS),
    ((1, 1, 128, 8, 1 << 24), UNS), ((1, (1 << 27) + 1, 16, 8, 8), UNS)])
def test_tables_shapes(call, shape, code):
    assert call(dflv.pages_desc(*shape)) == code


def test_tables_pointers():
    d = dflv.pages_desc(2, 4, 16, 8, 4)
    for k in ("n_past", "n_new", "n_held", "free_list", "n_free", "table", "slots", "status_dev"):
        assert grow(d, **{k: None}) == BAD and grow(d, **{k: 18}) == BAD, k
    for k in ("keep_len", "n_held", "free_list", "n_free", "table", "status_dev"):
        assert release(d, **{k: None}) == BAD and release(d, **{k: 18}) == BAD, k


KV = dict(B=2, N_max=4, Hkv=2, D=64, page=16, n_pages=8, kv_type=dflv.DFLV_KV_BF16)


def kv(**over):
    return dflv.paged_kv_desc(**{**KV, **over})


def append(d, **over):
    a = dict(slots=P, k_new=P, v_new=P, cache=dflv.dflv_kv_layer(P, P), status_dev=P)
    a.update(over)
    return dflv.dflv_paged_kv_append(d, stream=0, **a)


def commit(d, n=1, caches=None, **over):
    a = dict(slots=P, path=P, path_len=P, n_past=P, status_dev=P)
    a.update(over)
    return dflv.dflv_paged_kv_commit(d, n, caches or [dflv.dflv_kv_layer(P, P)] * n, stream=0, **a)


@pytest.mark.parametrize("call", [append, commit])
@pytest.mark.parametrize("over,code", [
    (dict(B=0), BAD), (dict(N_max=0), BAD), (dict(Hkv=0), BAD), (dict(D=0), BAD), (dict(n_pages=0), BAD),
    (dict(flags=2), BAD), (dict(kv_stride=64), BAD), (dict(kv_stride=132), BAD), (dict(kv_stride=-128), BAD),
    (dict(D=96), UNS), (dict(D=512), UNS), (dict(page=8), UNS), (dict(kv_type=dflv.DFLV_KV_Q8_0), UNS),
    (dict(kv_type=9), UNS), (dict(n_pages=1 << 27), UNS)])
def test_writes_shapes(call, over, code):
    assert call(kv(**over)) == code


def test_writes_pointers():
    for k in ("slots", "k_new", "v_new", "status_dev"):
        assert append(kv(), **{k: None}) == BAD and append(kv(), **{k: 18}) == BAD, k
    assert append(kv(), k_new=24) == BAD                       # 16-byte rows
    for c in (dflv.dflv_kv_layer(None, P), dflv.dflv_kv_layer(P, None), dflv.dflv_kv_layer(24, P)):
        assert append(kv(), cache=c) == BAD and commit(kv(), caches=[c]) == BAD
    for k in ("slots", "path", "path_len", "status_dev"):
        assert commit(kv(), **{k: None}) == BAD and commit(kv(), **{k: 18}) == BAD, k
    assert commit(kv(), n_past=18) == BAD
    assert commit(kv(N_max=65)) == UNS and commit(kv(), n=65) == UNS
    assert dflv.dflv_paged_kv_commit(kv(), 2, [dflv.dflv_kv_layer(P, P)], P, P, P, P, P, stream=0) == BAD
    assert dflv.dflv_paged_kv_commit(kv(), 0, [], P, P, P, P, P, stream=0) == BAD


AT = dict(B=2, N_max=4, Hq=4, Hkv=2, D=64, page=16, n_pages=8, max_pages=4, max_prefix_pages=4,
          kv_type=dflv.DFLV_KV_BF16, scale=0.125)


def at(**over):
    return dflv.prefix_attn_desc(**{**AT, **over})


def attn(d, **over):
    a = dict(prefix_table=P, prefix_len=P, table=P, parent=P, n_nodes=P, n_past=P, q=P,
             cache=dflv.dflv_kv_layer(P, P), out=P, status_dev=P, workspace=P, ws_bytes=1 << 40)
    a.update(over)
    return dflv.dflv_prefix_attn_verify(d, stream=0, **a)


@pytest.mark.parametrize("over,code", [
    (dict(B=0), BAD), (dict(N_max=0), BAD), (dict(Hq=0), BAD), (dict(Hkv=0), BAD), (dict(Hkv=3), BAD),
    (dict(max_pages=0), BAD), (dict(max_prefix_pages=0), BAD), (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(flags=1), BAD),
    (dict(q_stride=128), BAD), (dict(q_stride=260), BAD),
    (dict(N_max=65), UNS), (dict(B=1025), UNS), (dict(D=96), UNS), (dict(Hq=130), UNS), (dict(page=24), UNS),
    (dict(kv_type=dflv.DFLV_KV_F32), UNS), (dict(max_pages=1 << 26), UNS), (dict(max_prefix_pages=1 << 26), UNS)])
def test_attn_shapes(over, code):
    assert attn(at(**over)) == code
    assert dflv.dflv_prefix_attn_workspace_size(at(**over)) == 0


def test_attn_pointers():
    for k in ("prefix_table", "prefix_len", "table", "n_nodes", "n_past", "q", "out", "status_dev", "workspace"):
        assert attn(at(), **{k: None}) == BAD and attn(at(), **{k: 18}) == BAD, k
    for k in ("q", "out", "workspace"):
        assert attn(at(), **{k: 24}) == BAD
    assert attn(at(), parent=18) == BAD
    assert attn(at(), cache=dflv.dflv_kv_layer(P, 24)) == BAD
    need = dflv.dflv_prefix_attn_workspace_size(at())
    assert need > 0 and attn(at(), ws_bytes=need - 1) == CAP


def sample(d, tree=False, **over):
    a = dict(logits=P, temperature=P, top_k=P, top_p=P, min_p=P, u=P, n_nodes=P, drawn=P, logp=P, status_dev=P)
    if tree:
        a.update(tokens=P, parent=P, path=P, path_len=P, next_token=P)
    a.update(over)
    return (dflv.dflv_accept_sampled if tree else dflv.dflv_sample)(d, stream=0, **a)


@pytest.mark.parametrize("tree", [False, True])
def test_sample_refusals(tree):
    def d(B=2, N=4, V=100, kind=0, ld=0, flags=0):
        return dflv.sample_desc(B, N, V, kind, ld, flags)

    for bad in (d(B=0), d(N=0), d(V=0), d(ld=99), d(ld=-1), d(flags=1)):
        assert sample(bad, tree) == BAD
    for bad in (d(V=400001), d(kind=3), d(B=1 << 20, N=64)):
        assert sample(bad, tree) == UNS
    for k in ("logits", "temperature", "top_k", "top_p", "min_p", "u", "drawn", "status_dev"):
        assert sample(d(), tree, **{k: None}) == BAD and sample(d(), tree, **{k: 18}) == BAD, k
    assert sample(d(), tree, logits=24) == BAD
    assert sample(d(), tree, logp=18) == BAD and sample(d(), tree, n_nodes=18) == BAD
    if tree:
        assert sample(d(N=65), tree) == UNS
        for k in ("tokens", "parent", "n_nodes", "path", "path_len", "next_token"):
            assert sample(d(), tree, **{k: None}) == BAD and sample(d(), tree, **{k: 18}) == BAD, k


def test_tensors_that_do_not_fit_are_refused():
    # a host tensor, a wrong dtype, a short or a strided tensor never reach the library
    i = torch.zeros(64, dtype=torch.int32)
    assert grow(dflv.pages_desc(2, 4, 16, 8, 4), n_past=i) == BAD
    assert grow(dflv.pages_desc(2, 4, 16, 8, 4), n_past=i.long()) == BAD
    assert append(kv(), k_new=torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16)) == BAD
    assert append(kv(), cache=dflv.kv_layer(torch.zeros(4), torch.zeros(4))) == BAD
    assert attn(at(), q=torch.zeros(2, 4, 4, 64)) == BAD
    assert attn(at(), workspace=torch.zeros(4, dtype=torch.uint8), ws_bytes=1 << 20) == BAD
    assert sample(dflv.sample_desc(2, 4, 100), u=torch.zeros(8)) == BAD


# ------------------------------------------------------------------ pins of the oracle
def test_oracle_release_inverts_grow():
    rng = np.random.default_rng(5)
    B, N, page, width = 9, 40, 16, 7
    past = rng.integers(0, 60, B).astype(np.int32)
    new = rng.integers(0, N + 1, B).astype(np.int32)
    held = -(-past // page)
    ids = rng.permutation(B * width).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    used = 0
    for b in range(B):
        table[b, :held[b]] = ids[used:used + held[b]]
        used += held[b]
    free = np.concatenate([ids[used:], np.full(used, -1, np.int32)])
    h, nf, t, slots, st = paged.tables_grow(past, new, held, free, len(ids) - used, table, page, N)
    assert st == 0
    live = slots[slots >= 0]
    assert len(set(live.tolist())) == new.sum()               # no slot twice
    for b in range(B):
        for i in range(new[b]):
            assert slots[b, i] == t[b, (past[b] + i) // page] * page + (past[b] + i) % page
    assert sorted(t[b, j] for b in range(B) for j in range(h[b])) + sorted(free[:nf]) != []
    assert set(t[b, j] for b in range(B) for j in range(h[b])).isdisjoint(free[:nf].tolist())
    h2, free2, nf2, st = paged.tables_release(past, h, free, nf, t, page)
    assert st == 0 and nf2 == len(ids) - used and np.array_equal(h2, held) and np.array_equal(free2, free)


def test_oracle_attention_is_the_library_attention():
    # fp64 scaled_dot_product_attention over the gathered rows with an explicit mask
    rng = np.random.default_rng(6)
    B, N, Hq, Hkv, D, page, pre = 2, 5, 4, 2, 8, 16, 21
    k, v = rng.normal(size=(9, Hkv, page, D)), rng.normal(size=(9, Hkv, page, D))
    q = rng.normal(size=(B, N, Hq, D))
    tab, ptab = np.array([[3, 1], [0, 5]]), np.array([7, 2])
    parent = np.array([[-1, 0, 0, 1, 2], [-1, 0, 1, 2, 3]])
    past, n = np.array([17, 3]), np.array([5, 4])
    out, _ = paged.prefix_attn(ptab, pre, tab, parent, n, past, q, k, v, 0.3)
    for b in range(B):
        flat = lambda x, t, m: x[t].transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:m]  # noqa: E731
        kk = np.concatenate([flat(k, ptab, pre), flat(k, tab[b], past[b] + n[b])])
        vv = np.concatenate([flat(v, ptab, pre), flat(v, tab[b], past[b] + n[b])])
        mask = np.ones((n[b], len(kk)), bool)
        for i in range(n[b]):
            for j in range(n[b]):
                a = i
                while a > j:
                    a = parent[b, a]
                mask[i, pre + past[b] + j] = a == j
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x.transpose(1, 0, 2)))  # noqa: E731
        ref = torch.nn.functional.scaled_dot_product_attention(
            t(q[b, :n[b]]), t(kk).repeat_interleave(2, 0), t(vv).repeat_interleave(2, 0),
            attn_mask=torch.from_numpy(mask), scale=0.3)
        assert np.allclose(out[b, :n[b]], ref.numpy().transpose(1, 0, 2), atol=1e-12)


def test_oracle_sampling():
    x = [1.0, 3.0, 2.0, 3.0, -math.inf, 0.0]
    w = np.exp(np.array(x) - 3)
    draw = lambda u, T=1.0, k=0, p=1.0, m=0.0: paged.sample_row(x, T, k, p, m, u)[0]  # noqa: E731
    run = np.cumsum(w) / w.sum()
    for u in np.linspace(0, 0.999, 50):
        assert draw(u) == int(np.searchsorted(run, u, side="right"))
    assert {draw(u, k=1) for u in np.linspace(0, 0.99, 20)} == {1}          # tie: the lower index
    assert {draw(u, k=3) for u in np.linspace(0, 0.99, 50)} == {1, 2, 3}
    assert {draw(u, p=0.0) for u in np.linspace(0, 0.99, 20)} == {1}
    assert {draw(u, p=1 / w.sum()) for u in np.linspace(0, 0.99, 20)} == {1}
    assert {draw(u, p=1.01 / w.sum()) for u in np.linspace(0, 0.99, 20)} == {1, 3}
    assert {draw(u, m=0.3) for u in np.linspace(0, 0.99, 50)} == {1, 2, 3}
    assert draw(0.9, T=0.0) == 1
    assert paged.sample_row(x, -1.0, 0, 1.0, 0.0, 0.5)[3] == paged.DEV_SAMPLE
    assert paged.sample_row([-math.inf] * 4, 1.0, 0, 1.0, 0.0, 0.5)[::3] == (0, paged.DEV_SAMPLE)


@pytest.mark.parametrize("scale,code", [(3e38, UNS), (-3e38, UNS), (2.0 ** 127, CAP), (-(2.0 ** 127), CAP), (0.0, CAP)])
def test_attn_scales(scale, code):
    # beyond 2^127 the scale times log2(e) is not finite (CAP: what comes after the
    # descriptor, a workspace of no bytes)
    assert attn(at(scale=scale), ws_bytes=0) == code


@pytest.mark.parametrize("shape", [(0, 4, 2, 64), (2, 0, 2, 64), (0, 0, 2, 64)])
def test_rows_of_an_empty_tensor_are_refused(shape):
    # with a stride of their own, whatever the descriptor says
    x = torch.empty(shape, dtype=torch.bfloat16)
    for B, N in ((0, 0), shape[:2], (2, 4)):
        with pytest.raises(dflv._Refused):
            dflv._rows(x, (torch.bfloat16,), B, N, 128, 256, x.get_device())


@pytest.mark.parametrize("call,first", [(grow, "n_past"), (release, "keep_len")])
def test_tables_of_too_many_sequences_are_refused(call, first):
    # whose sums would take the GPU minutes and more (BAD: the NULL that comes
    # after the descriptor)
    for B, code in ((1 << 20, BAD), ((1 << 20) + 1, UNS), (1 << 30, UNS)):
        assert call(dflv.pages_desc(B, 1, 16, 8, 1), **{first: None}) == code
