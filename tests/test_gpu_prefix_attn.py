"""GPU parity of the shared-prefix attention against the fp64 oracle.

Tolerance, element by element, from the roundings the call documents, with
u = eps / 2 of the 16-bit type and A = the oracle's sum of p |v|:
  * the weights are rounded to the type before the product with V: u A
    (fp16 weights also lose up to 2^-25 of the largest each where they are
    subnormal; the kernel scales them up by 2^6: keys 2^-31 max|v|);
  * the output is rounded once: u |ref|;
  * fp32 scores: q.k over D terms errs by D 2^-24 sum|q k| scale at most, and a
    score error e changes weights by a factor e^e.  With |q| ~ 1.5, |k| ~ 1
    normal, sum|q k| scale <= 1.2 sqrt(D), so 2 e <= 2.4 D sqrt(D) 2^-24 (6e-4
    at D = 256), the running rescales and sums a few 2^-24 more: 2^-10 A covers
    both in bf16 (a quarter of u), and the same holds against u = 2^-11 in
    fp16, where 2 e A is added in full."""
import math

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


TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


class Case:
    def __init__(self, seed, B, N, Hq, Hkv, D, page, kind, prefix, past, n, chain=False, poison=True, n_pages=None):
        rng = np.random.default_rng(seed)
        self.__dict__.update(B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, page=page, kind=kind, prefix=prefix)
        self.past, self.n = np.asarray(past, np.int32), np.asarray(n, np.int32)
        t = TYPES[kind]
        self.t = t
        pre = max(1, -(-prefix // page))
        width = max(1, int(max(-(-(int(p) + int(m)) // page) for p, m in zip(self.past, self.n))))
        need = pre + B * width
        self.n_pages = n_pages or need + 2
        ids = (rng.permutation(need + 2) + self.n_pages - need - 2).astype(np.int32)
        self.ptab, self.tab = ids[:pre].copy(), ids[pre:pre + B * width].reshape(B, width).copy()
        self.parent = np.maximum(np.arange(N)[None] - rng.integers(1, 5, (B, N)), 0).astype(np.int32)
        self.parent[:, 0] = -1
        if chain:
            self.parent = np.tile(np.arange(-1, N - 1, dtype=np.int32), (B, 1))
        self.q = torch.from_numpy(rng.normal(size=(B, N, Hq, D)) * 1.5).to(t)
        small = (need + 2, Hkv, page, D)
        self.k, self.v = (torch.from_numpy(rng.normal(size=small)).to(t) for _ in range(2))
        self.first = self.n_pages - need - 2
        if poison:
            # what no sequence has written: NaN and infinities
            live = torch.zeros((need + 2, page), dtype=torch.bool)
            for tab, length in [(self.ptab, prefix)] + [(self.tab[b], int(self.past[b] + self.n[b])) for b in range(B)
                                                        if self.n[b]]:
                for j in range(length):
                    live[tab[j // page] - self.first, j % page] = True
            mask = ~live[:, None, :, None].expand(small)
            self.k[mask] = float("nan")
            self.v[mask] = float("inf")
            self.v[:, :, ::2][mask[:, :, ::2]] = float("nan")

    def planes(self):
        if self.first == 0:
            return self.k.cuda(), self.v.cuda()
        out = []
        for x in (self.k, self.v):
            y = torch.empty((self.n_pages,) + tuple(x.shape[1:]), dtype=self.t, device="cuda")
            y[self.first:] = x.cuda()
            out.append(y)
        return out

    def oracle(self, n=None):
        f = lambda x: x.double().numpy()  # noqa: E731
        with np.errstate(invalid="ignore", over="ignore"):
            return paged.prefix_attn(self.ptab - self.first, self.prefix, self.tab - self.first, self.parent,
                                     self.n if n is None else n, self.past, f(self.q), f(self.k), f(self.v),
                                     1 / math.sqrt(self.D))

    def desc(self, dflv, q_stride=0):
        return dflv.prefix_attn_desc(self.B, self.N, self.Hq, self.Hkv, self.D, self.page, self.n_pages,
                                     self.tab.shape[1], len(self.ptab),
                                     dflv.DFLV_KV_BF16 if self.kind == "bf16" else dflv.DFLV_KV_F16,
                                     1 / math.sqrt(self.D), q_stride)

    def run(self, dflv, parent="given", q=None, q_stride=0, stream=None, planes=None, **over):
        a = dict(ptab=self.ptab, plen=np.array([self.prefix], np.int32), tab=self.tab, n=self.n, past=self.past)
        a.update(over)
        d = {k: dev(np.asarray(v, np.int32)) for k, v in a.items()}
        par = None if parent is None else dev(self.parent if isinstance(parent, str) else parent)
        kp, vp = planes or self.planes()
        out = torch.full((self.B, self.N, self.Hq, self.D), -7.0, dtype=self.t, device="cuda")
        desc = self.desc(dflv, q_stride)
        size = dflv.dflv_prefix_attn_workspace_size(desc)
        ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")   # NaN: its contents do not matter
        st = zeros_status()
        dflv.check(dflv.dflv_prefix_attn_verify(desc, d["ptab"], d["plen"], d["tab"], par, d["n"], d["past"],
                                                self.q.cuda() if q is None else q, dflv.kv_layer(kp, vp), out, st, ws,
                                                size, stream=stream))
        torch.cuda.synchronize()
        return out, int(st)

    def compare(self, out, ref=None):
        ref, mag = self.oracle() if ref is None else ref
        got = out.double().cpu().numpy()
        live = np.arange(self.N)[None] < self.n[:, None]
        assert (got[~live] == -7).all()
        u = torch.finfo(self.t).eps / 2
        g, r, a = got[live], ref[live], mag[live]
        tol = u * (a + np.abs(r)) + 2.0 ** -10 * a * (u / 2.0 ** -8)
        if self.kind == "f16":
            vmax = float(self.v[torch.isfinite(self.v)].abs().max())
            tol += (self.prefix + int(self.past.max()) + self.N) * 2.0 ** -31 * vmax
            tol += 2.4 * self.D * math.sqrt(self.D) * 2.0 ** -24 * a
        bad = ~(np.abs(g - r) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:5], g[bad][:5], r[bad][:5], (np.abs(g - r) / tol)[bad].max())


SHAPES = [
    # B, N, Hq, Hkv, D, page, prefix, past, n
    (1, 1, 1, 1, 64, 16, 0, [0], [1]),                       # one token, nothing before it
    (1, 1, 1, 1, 128, 16, 1, [0], [1]),
    (1, 1, 6, 1, 256, 16, 64, [0], [1]),
    (2, 1, 4, 2, 64, 32, 63, [0, 65], [1, 1]),
    (3, 1, 24, 4, 256, 16, 130, [1, 63, 64], [1, 1, 1]),
    (4, 1, 32, 8, 128, 128, 1000, [7, 0, 300, 129], [1, 0, 1, 1]),
    (2, 7, 6, 2, 128, 16, 200, [40, 61], [7, 3]),
    (3, 22, 24, 4, 256, 64, 300, [100, 0, 42], [22, 5, 0]),
    (2, 64, 12, 2, 256, 16, 65, [33, 127], [64, 50]),        # trees over several key tiles
    (2, 64, 8, 8, 64, 32, 129, [500, 2], [64, 1]),
    (2, 64, 64, 1, 64, 16, 100, [10, 20], [64, 33]),         # 4096 rows of one head
    (1, 33, 64, 1, 128, 64, 0, [77], [33]),                  # no prefix
    (5, 3, 5, 5, 64, 16, 17, [0, 0, 0, 0, 0], [3, 2, 1, 0, 3]),
    (2, 13, 8, 8, 64, 16, 1017, [333, 200], [13, 9]),
    (40, 2, 8, 2, 128, 32, 512, list(range(0, 400, 10)), [1, 2] * 20),
    (1, 4, 6, 2, 128, 128, 9000, [0], [4]),                  # a long prefix for few rows
    (1, 1, 8, 4, 256, 64, 2, [12000], [1]),                  # a long sequence, a short prefix
]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_parity(dflv, shape, kind):
    B, N, Hq, Hkv, D, page, prefix, past, n = shape
    c = Case(B * N + D, B, N, Hq, Hkv, D, page, kind, prefix, past, n)
    out, st = c.run(dflv)
    assert st == 0
    c.compare(out)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("edge", [-1, 0, 1])
def test_tile_and_page_edges(dflv, D, page, edge):
    # prefix, past and past + n on, before and behind multiples of 64 and of the page
    c = Case(D + page + edge, 4, 3, 4, 2, D, page, "bf16", 128 + edge, [64 + edge, 61 + edge, 128 + edge, 125 + edge],
             [3, 3, 1, 3])
    out, st = c.run(dflv)
    assert st == 0
    c.compare(out)


def test_chains_without_a_parent_array(dflv):
    c = Case(4, 3, 9, 6, 2, 128, 16, "bf16", 70, [5, 60, 0], [9, 8, 1], chain=True)
    ref = c.oracle()
    for parent in (None, "given"):
        out, st = c.run(dflv, parent=parent)
        assert st == 0
        c.compare(out, ref)


def test_strided_queries(dflv):
    c = Case(5, 2, 6, 4, 2, 64, 16, "f16", 40, [20, 3], [6, 4])
    wide = torch.randn(2, 6, 4 * 64 + 512).half().cuda()
    wide[:, :, 256:512] = c.q.flatten(2).cuda()
    q = wide[:, :, 256:512].unflatten(2, (4, 64))
    out, st = c.run(dflv, q=q, q_stride=4 * 64 + 512)
    assert st == 0
    c.compare(out)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_values_of_other_branches_do_not_leak(dflv, value):
    # node 2's value row is not finite: only its descendants may see it
    c = Case(6, 2, 8, 4, 2, 128, 16, "bf16", 33, [62, 10], [8, 6])
    ref, mag = c.oracle()
    at = c.past + 2
    for b in range(2):
        c.v[c.tab[b, at[b] // 16], :, at[b] % 16, ::3] = value
    out, st = c.run(dflv)
    assert st == 0
    got = out.double().cpu().numpy()
    for b in range(2):
        for i in range(int(c.n[b])):
            a = i
            while a > 2:
                a = int(c.parent[b, a])
            hit = got[b, i, :, ::3]
            if a == 2:
                assert (np.isnan(hit) if math.isnan(value) else hit == value).all()
            else:
                assert np.isfinite(got[b, i]).all()
                u = 2.0 ** -8
                assert (np.abs(got[b, i] - ref[b, i]) <= u * (mag[b, i] + np.abs(ref[b, i])) + 2.0 ** -10 * mag[b, i]).all()


def test_large_and_equal_scores(dflv):
    # scores of several hundred: the running maximum has to follow them
    c = Case(8, 2, 3, 4, 2, 64, 16, "bf16", 300, [100, 5], [3, 3])
    c.q *= 40
    ref, mag = c.oracle()
    out, st = c.run(dflv)
    got = out.double().cpu().numpy()
    # score errors grow with the scores: D 2^-24 sum|q k| scale, 40 times the usual
    tol = 2.0 ** -8 * (mag + np.abs(ref)) + 40 * 2.4 * 64 * 8 * 2.0 ** -24 * mag + 2.0 ** -10 * mag
    live = np.arange(3)[None] < c.n[:, None]
    assert st == 0 and (np.abs(got - ref)[live] <= tol[live]).all()
    c.k[:] = 0.5                     # all scores equal: the mean of the values
    c.v = torch.where(torch.isfinite(c.v), c.v, 0)
    out, st = c.run(dflv)
    c.compare(out)


def test_bad_inputs_raise_their_bits(dflv):
    c = Case(9, 2, 4, 4, 2, 64, 16, "bf16", 40, [20, 20], [4, 4], poison=False)
    ref = c.oracle()

    def good(out, b):
        u = 2.0 ** -8
        g = out.double().cpu().numpy()[b]
        assert (np.abs(g - ref[0][b]) <= u * (ref[1][b] + np.abs(ref[0][b])) + 2.0 ** -10 * ref[1][b]).all()

    for n, bits in (([5, 4], dflv.DFLV_DEV_TOPOLOGY), ([-1, 4], dflv.DFLV_DEV_TOPOLOGY)):
        out, st = c.run(dflv, n=n)
        assert st == bits
        good(out, 1)
    for past in (-1, 29, 1 << 30):
        out, st = c.run(dflv, past=[past, 20])
        assert st == dflv.DFLV_DEV_CAPACITY
        good(out, 1)
    for plen in (-1, 49, 1 << 30):
        out, st = c.run(dflv, plen=[plen])
        assert st == dflv.DFLV_DEV_CAPACITY
    par = c.parent.copy()
    for bad in ([-1, 1, 1, 2], [0, 0, 1, 2], [-1, 0, 5, 2], [-1, 0, -1, 2]):
        par[0] = bad
        out, st = c.run(dflv, parent=par)
        assert st == dflv.DFLV_DEV_TOPOLOGY
        good(out, 1)
    for tab in ("tab", "ptab"):
        for page in (-1, c.n_pages, 1 << 30):
            x = (c.tab if tab == "tab" else c.ptab).copy()
            x.flat[0] = page
            out, st = c.run(dflv, **{tab: x})
            assert st == dflv.DFLV_DEV_PAGE
            if tab == "tab":
                good(out, 1)


def test_pool_past_32_bits(dflv):
    # 2.7e9 elements a plane: the pages in use lie at its end
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    c = Case(10, 2, 5, 8, 4, 256, 64, "bf16", 100, [70, 3], [5, 2], n_pages=41000)
    out, st = c.run(dflv)
    assert st == 0
    c.compare(out)


def test_results_do_not_depend_on_the_call(dflv):
    # the same call on two streams at once (a workspace each), again and again,
    # and captured and replayed with other lengths
    c = Case(11, 6, 5, 12, 2, 128, 16, "bf16", 700, [10, 200, 3, 64, 0, 90], [5, 1, 5, 2, 3, 4])
    ref, st = c.run(dflv)
    assert st == 0
    c.compare(ref)
    planes = c.planes()
    desc, size = c.desc(dflv), dflv.dflv_prefix_attn_workspace_size(c.desc(dflv))
    a = [dev(np.asarray(x, np.int32)) for x in (c.ptab, [c.prefix], c.tab, c.parent, c.n, c.past)]
    q, kv = c.q.cuda(), dflv.kv_layer(*planes)
    lanes = []
    for _ in range(2):
        lanes.append((torch.cuda.Stream(), torch.empty(size, dtype=torch.uint8, device="cuda"),
                      torch.full_like(ref, -7.0)))
    st = zeros_status()
    torch.cuda.synchronize()
    for _ in range(10):
        for s, ws, out in lanes:
            dflv.check(dflv.dflv_prefix_attn_verify(desc, *a, q, kv, out, st, ws, size, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(out, ref) for _, _, out in lanes) and int(st) == 0
    g = torch.cuda.CUDAGraph()
    _, ws, out = lanes[0]
    with torch.cuda.graph(g):
        dflv.check(dflv.dflv_prefix_attn_verify(desc, *a, q, kv, out, st, ws, size))
    for prefix, n in ((700, c.n), (33, c.n), (700, np.array([1, 1, 0, 1, 1, 1], np.int32))):
        a[1].fill_(prefix)
        a[4].copy_(dev(n))
        out.fill_(-7.0)
        g.replay()
        torch.cuda.synchronize()
        full, c.prefix, keep, c.n = c.prefix, prefix, c.n, n
        fresh, _ = c.run(dflv)
        assert torch.equal(out, fresh)
        c.prefix, c.n = full, keep
    assert int(st) == 0


@pytest.mark.parametrize("shape", [(2, 4, 4, 2, 64, 16, 40, [20, 20], [4, 3]), (2, 4, 6, 2, 128, 16, 300, [0, 70], [4, 4]),
                                   (3, 40, 12, 2, 256, 64, 0, [130, 9, 60], [33, 40, 40]),
                                   (700, 3, 2, 1, 64, 16, 33, [5] * 700, [3] * 700)])
def test_a_malformed_tree_takes_no_part(dflv, shape):
    B, N, Hq, Hkv, D, page, prefix, past, n = shape
    c = Case(14, B, N, Hq, Hkv, D, page, "bf16", prefix, past, n)
    ref = c.oracle()
    good = c.parent.copy()
    for b in {0, B - 1, B // 2}:
        last = int(c.n[b]) - 1
        for at, value in ((0, 0), (0, -2), (1, -1), (1, 1), (last, last), (last, 1 << 30)):
            par = good.copy()
            par[b, at] = value
            out, st = c.run(dflv, parent=par)
            assert st == dflv.DFLV_DEV_TOPOLOGY
            assert (out[b] == -7).all()
            n0, c.n = c.n, c.n.copy()
            c.n[b] = 0
            c.compare(out, ref)
            c.n = n0
    # what stands behind a tree's nodes, or in a sequence without any, is not looked at
    par = good.copy()
    for b in range(B):
        par[b, int(c.n[b]):] = 1 << 20
    out, st = c.run(dflv, parent=par)
    assert st == 0
    c.compare(out, ref)


class Scaled(Case):
    scale = 0.0

    def desc(self, dflv, q_stride=0):
        d = super().desc(dflv, q_stride)
        d.scale = self.scale
        return d

    def oracle(self, n=None):
        f = lambda x: x.double().numpy()  # noqa: E731
        with np.errstate(invalid="ignore", over="ignore"):
            return paged.prefix_attn(self.ptab - self.first, self.prefix, self.tab - self.first, self.parent,
                                     self.n if n is None else n, self.past, f(self.q), f(self.k), f(self.v),
                                     float(np.float32(self.scale)))


SCALED = [(3, 5, 6, 2, 64, 16, 130, [20, 63, 0], [5, 1, 4]), (2, 40, 12, 2, 128, 16, 200, [40, 61], [40, 30]),
          (3, 22, 24, 4, 256, 64, 300, [100, 0, 42], [22, 5, 0])]


@pytest.mark.parametrize("shape", SCALED)
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [-1.0, -0.25, 0.0, -0.0, 1e-20, -1e-35, 2.0 ** -149])
def test_scales_of_either_sign_and_none(dflv, shape, kind, scale):
    # (-1 and -0.25: as parts of 1 / sqrt(D), for which the tolerance is derived)
    B, N, Hq, Hkv, D, page, prefix, past, n = shape
    c = Scaled(15, B, N, Hq, Hkv, D, page, kind, prefix, past, n)
    c.scale = scale / math.sqrt(D) if scale <= -0.25 else scale
    out, st = c.run(dflv)
    assert st == 0
    c.compare(out)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale,factor", [(0.0, 2.0 ** 100), (1e-35, 2.0 ** 110), (-2.0 ** -120, 2.0 ** 114)])
def test_scales_that_undo_large_scores(dflv, D, scale, factor):
    # products of queries and keys of up to 2^120: none of their size is left in
    # the weights
    c = Scaled(16, 3, 5, 6, 2, D, 16, "bf16", 130, [20, 63, 0], [5, 1, 4])
    c.q = (c.q.float() * (factor / 2.0 ** 60)).bfloat16()
    c.k = torch.where(torch.isfinite(c.k), c.k.float() * 2.0 ** 60, c.k.float()).bfloat16()
    c.scale = scale
    out, st = c.run(dflv)
    assert st == 0
    c.compare(out)


def test_equal_scores_and_their_status(dflv):
    c = Case(17, 2, 3, 4, 2, 64, 16, "bf16", 300, [100, 5], [3, 3])
    c.k[:] = 0.5                     # all scores of a row equal: the mean of the values
    out, st = c.run(dflv)
    assert st == 0
    c.compare(out)
