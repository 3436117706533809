"""GPU parity of tree attention with a 64-bit implementation, over pages,
rectangles, GATHER groups and pools: types, head layouts, lengths, tile and page
edges, strides, values that are not finite in places that take no part, status
bits, cache offsets past 4 GiB, workspaces in turn, streams and graphs."""
import math

import numpy as np
import pytest
import torch

from tests import tree_oracle as T
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NAN = float("nan")


@pytest.fixture(scope="module")
def sd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ragged_kv_realignment_amd as m
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """One call's inputs on the device and each row's old keys and values on the CPU.  Everything that takes no part is NaN."""

    def __init__(self, sd, seed, dt, store, lens, N, H, G, Dh, page=16, L=2, layer=1, used=None, wide=False, spread=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.B, self.N, self.H, self.G, self.Dh, self.dt, self.L, self.layer = len(lens), N, H, G, Dh, dt, L, layer
        B = self.B

        def normal(*shape):
            return torch.randn(shape, generator=g).mul_(spread).to(dt)

        self.old = [(normal(H, n, Dh), normal(H, n, Dh)) for n in lens]
        used = [N] * B if used is None else used
        self.parent = np.stack([T.random_tree(rng, N, used[b], wide) for b in range(B)])
        self.q = normal(B, N, H * G, Dh)
        self.kv_new = torch.full((L, 2, B, H, N, Dh), NAN, dtype=dt)
        self.kv_new[layer] = normal(2, B, H, N, Dh)
        for b in range(B):
            self.q[b, used[b]:] = NAN
            self.kv_new[layer, :, b, :, used[b]:] = NAN
        self.rows, self.group = None, 0
        if store == "paged":
            rows = B + 2
            self.rows = rng.permutation(rows)[:B].astype(np.int32)
            blocks = max(1, max(-(-n // page) for n in lens)) + 1
            n_pages = sum(-(-n // page) for n in lens) + 3
            order = rng.permutation(n_pages)
            pages = torch.full((L, 2, n_pages, H, page, Dh), NAN, dtype=dt)
            table = np.full((rows, blocks), -1, np.int32)
            ln, at = np.zeros(rows, np.int32), 0
            for b, n in enumerate(lens):
                ln[self.rows[b]] = n
                for k in range(-(-n // page)):
                    pg = order[at]
                    at += 1
                    table[self.rows[b], k] = pg
                    m = min(page, n - k * page)
                    for j in (0, 1):
                        pages[layer, j, pg, :, :m] = self.old[b][j][:, k * page:k * page + m]
            z = torch.zeros(1, dtype=torch.int32, device="cuda")
            self.cache = sd.PagedKV(pages.cuda(), dev(table), torch.zeros(n_pages, dtype=torch.int32, device="cuda"), z,
                                    torch.zeros((rows, blocks * page), dtype=torch.int32, device="cuda"), dev(ln))
        else:
            cap = max(lens) + 5
            width = None
            if store == "group":  # rectangles of two rows, each as wide as its longer row
                self.group = 2
                width = np.array([max(lens[k:k + 2]) for k in range(0, B, 2)], np.int32)
            elif store == "rect":
                width = np.array([max(lens) + 3], np.int32)
            rows = B
            where = np.arange(B)
            if store == "pool":
                rows = B + 3
                where = self.rows = rng.permutation(rows)[:B].astype(np.int32)
            kv = torch.full((L, 2, rows, H, cap, Dh), NAN, dtype=dt)
            ln = np.zeros(rows, np.int32)
            for b, n in enumerate(lens):
                s = 0 if width is None else width[b // 2 if self.group else 0] - n
                ln[where[b]] = n
                for j in (0, 1):
                    kv[layer, j, where[b], :, s:s + n] = self.old[b][j]
            self.cache = sd.SeqBuf(kv.cuda(), torch.zeros((rows, cap), dtype=torch.int32, device="cuda"), dev(ln),
                                   width=None if width is None else dev(width))
        self.scale = Dh ** -0.5

    def call(self, sd, q=None, out=None, **kw):
        q = self.q.cuda() if q is None else q
        rows = None if self.rows is None else dev(self.rows)
        return sd.tree_attention(q, self.cache, self.layer, self.kv_new.cuda(), dev(self.parent), rows=rows, group=self.group,
                                 out=out, **kw)

    def want(self, out, scale=None):
        return T.attention(self.q, self.old, self.kv_new[self.layer], self.parent, self.scale if scale is None else scale, out)

    def check(self, sd, **kw):
        out = torch.full((self.B, self.N, self.H * self.G, self.Dh), 7.0, dtype=self.dt)
        want, tol = self.want(out, kw.get("scale"))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = self.call(sd, out=out.cuda(), status=st, **kw)
        torch.cuda.synchronize()
        assert int(st) == 0
        off = (got.cpu().double() - want).abs()
        assert bool((off <= tol).all()), (float((off - tol).max()), float(off.max()))
        return got


CASES = [
    # dtype, store, lens, N, H, G, Dh, page
    (BF16, "paged", [1], 1, 1, 1, 64, 16), (BF16, "paged", [0], 1, 2, 4, 128, 16), (F16, "rect", [0, 5], 3, 2, 2, 64, 0),
    (BF16, "paged", [31, 32, 33, 0, 127, 128, 129], 5, 2, 4, 128, 16), (F16, "paged", [64, 1, 95], 17, 3, 1, 80, 5),
    (F32, "paged", [40, 7], 6, 2, 3, 64, 1), (F32, "rect", [200, 3, 64], 13, 2, 2, 128, 0), (F32, "pool", [100, 45], 9, 1, 4, 256, 0),
    (BF16, "rect", [300, 17, 150], 24, 2, 4, 128, 0), (BF16, "group", [70, 33, 9, 129, 20], 7, 2, 5, 96, 0),
    (F16, "pool", [130, 0, 77, 256], 33, 1, 2, 64, 0), (BF16, "paged", [500, 90], 64, 1, 4, 128, 64),
    (BF16, "paged", [77, 200], 40, 2, 3, 128, 24), (F16, "paged", [150, 31], 64, 1, 7, 64, 7), (BF16, "rect", [90, 64], 96, 1, 2, 256, 0),
    (BF16, "paged", [129], 256, 1, 1, 128, 16), (F16, "rect", [60], 200, 1, 3, 8, 0), (F32, "paged", [33, 200], 70, 1, 2, 16, 16),
    (F32, "rect", [65], 50, 1, 3, 32, 0), (BF16, "paged", [40], 3, 1, 16, 248, 16), (BF16, "pool", [64, 10], 32, 8, 1, 128, 0),
    (F32, "paged", [50], 130, 1, 2, 256, 3), (F16, "paged", [70], 48, 2, 1, 256, 16),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(sd, case):
    dt, store, lens, N, H, G, Dh, page = CASES[case]
    say("tree attention", CASES[case])
    used = [max(1, N - 3 * b) for b in range(len(lens))]
    Case(sd, 200 + case, dt, store, lens, N, H, G, Dh, page, used=used, wide=case % 2 == 0).check(sd)


@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_attention_random(sd, dt):
    rng = np.random.default_rng(7)
    ws = {}
    for k in range(12):
        store = ["paged", "rect", "pool", "group"][k % 4]
        B, N = int(rng.integers(1, 9)), int(rng.integers(1, 40))
        H, G = int(rng.integers(1, 4)), int(rng.integers(1, 9))
        Dh = int(rng.choice([64, 128, 256, 32, 96, 200]))
        lens = [int(x) for x in rng.integers(0, 400, B)]
        page = int(rng.choice([1, 3, 16, 64]))
        say("random attention", dt, store, lens, N, H, G, Dh, page)
        c = Case(sd, 300 + k, dt, store, lens, N, H, G, Dh, page, L=1, layer=0, spread=1.7,
                 used=[int(rng.integers(1, N + 1)) for _ in range(B)])
        key = (N, G, Dh)
        ws.setdefault(key, sd.tree_attention_workspace(B, N, H * G, H, Dh))
        a = c.check(sd, ws=ws[key])
        assert torch.equal(a, c.check(sd, ws=ws[key]))  # the same bytes again, the counters cleared
        assert torch.equal(a, c.check(sd))
        c.check(sd, scale=-0.3)


@pytest.mark.parametrize("dt,H,G,Dh,N", [(BF16, 1, 4, 128, 6), (F16, 2, 1, 64, 1), (BF16, 2, 16, 128, 20), (F32, 1, 2, 128, 3),
                                         (BF16, 1, 8, 256, 4)])
def test_attention_long_rows_split(sd, dt, H, G, Dh, N):
    """Long rows beside short ones: segments over many workgroups, joined by the last to arrive."""
    say("long rows", dt, H, G, Dh, N)
    c = Case(sd, 17, dt, "paged", [9000, 3, 20011, 0], N, H, G, Dh, 16, L=1, layer=0)
    ws = sd.tree_attention_workspace(4, N, H * G, H, Dh)
    first = c.check(sd, ws=ws)
    for _ in range(5):
        assert torch.equal(first, c.call(sd, out=torch.full_like(first, 7.0), ws=ws))


def test_attention_strides_and_fused_projection(sd):
    c = Case(sd, 23, BF16, "paged", [50, 200], 11, 2, 4, 128)
    want = c.check(sd)
    qkv = torch.full((2, 13, 8 + 4 + 3, 128), NAN, dtype=BF16, device="cuda")
    q = qkv[:, 1:12, 2:10]
    q.copy_(c.q)
    wide = torch.full((2, 8, 12, 160), 7.0, dtype=BF16, device="cuda")  # heads before nodes, a gap after each head
    out = wide[:, :, :11, 16:144].transpose(1, 2)
    c.call(sd, q=q, out=out)
    assert torch.equal(out, want)
    out.fill_(7.0)
    assert bool((wide == 7.0).all())


def test_attention_large_scores_and_one_hot(sd):
    """Scores of hundreds: one key takes all the weight; the running maximum rises often."""
    for dt in (BF16, F16, F32):
        c = Case(sd, 29, dt, "rect", [700, 64], 5, 2, 2, 64, L=1, layer=0, spread=5.0)
        c.check(sd, scale=0.5)


@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_attention_values_that_are_not_finite(sd, dt):
    """A branch whose entries overflowed reaches itself and its descendants only."""
    N, H, G, Dh = 40, 2, 3, 64
    c = Case(sd, 31, dt, "paged", [45, 0], N, H, G, Dh, L=1, layer=0)
    parent = np.full(N, -1, np.int32)
    parent[1:] = [0, 0] + [max(1, i - 2) for i in range(3, N)]  # two branches: odd nodes under 1, even under 2
    c.parent[:] = parent
    c.kv_new[0, 1, 0, 0, 5, 3] = float("inf")
    c.kv_new[0, 1, 0, 0, 37, 10] = -float("inf")
    c.kv_new[0, 1, 0, 1, 8, :] = NAN
    c.kv_new[0, 0, 1, 0, 7, 0] = float("inf")
    c.kv_new[0, 0, 1, 1, 4, :] = NAN
    c.kv_new[0, 1, 1, 1, 0, 63] = float("inf")  # the root's: everybody's
    out = torch.full((2, N, H * G, Dh), 7.0, dtype=dt)
    got = c.call(sd, out=out.cuda()).cpu().double()
    clean = c.kv_new.clone()
    c.kv_new = torch.where(torch.isfinite(clean), clean, torch.zeros_like(clean))
    want, tol = c.want(out)
    lines = T.lines(parent)
    for i in range(N):
        has = set(lines[i])
        w = want[:, i].clone()
        if 5 in has:
            w[0, :G, 3] = float("inf")
        if 37 in has:
            w[0, :G, 10] = -float("inf")
        if 8 in has:
            w[0, G:] = NAN
        if 4 in has:
            w[1, G:] = NAN
        else:
            w[1, G:, 63] = float("inf")
        skip = 7 in has  # an infinite key: the score is +-inf or NaN by the query's sign
        a, b, t = got[:, i], w, tol[:, i]
        if skip:
            a, b, t = torch.cat([a[0], a[1, G:]]), torch.cat([b[0], b[1, G:]]), torch.cat([t[0], t[1, G:]])
        fine = torch.isfinite(b)
        assert bool(((a - b).abs()[fine] <= t[fine]).all()), i
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a[~fine & ~torch.isnan(b)], b[~fine & ~torch.isnan(b)]), i


def test_attention_rows_listed_twice(sd):
    c = Case(sd, 37, F16, "paged", [33, 90], 4, 1, 2, 64)
    c.rows = np.array([c.rows[1], c.rows[1]], np.int32)
    c.old = [c.old[1], c.old[1]]
    c.check(sd)


def test_attention_status(sd):
    base = Case(sd, 41, BF16, "paged", [20, 40], 4, 1, 2, 64)
    for what in ("row", "negative row", "length", "negative length"):
        c = Case(sd, 41, BF16, "paged", [20, 40], 4, 1, 2, 64)
        if what == "row":
            c.rows[1] = 4
        elif what == "negative row":
            c.rows[0] = -1
        else:
            c.cache.len[int(c.rows[0])] = -1 if what[0] == "n" else c.cache.tokens.shape[1] + 1
        out = torch.full((2, 4, 2, 64), 7.0, dtype=BF16, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.call(sd, out=out, status=st)
        assert int(st) == sd.S_LEN_RANGE and bool((out == 7.0).all()), what
    c = Case(sd, 43, BF16, "rect", [20, 40], 4, 1, 2, 64)
    c.cache.width[0] = 39  # shorter than a row
    out = torch.full((2, 4, 2, 64), 7.0, dtype=BF16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.call(sd, out=out, status=st)
    assert int(st) == sd.S_LEN_RANGE and bool((out == 7.0).all())
    # a bad page: its positions take no part, the others do
    for bad in (-1, base.cache.pages.shape[2], 1 << 30):
        c = Case(sd, 41, BF16, "paged", [20, 40], 4, 1, 2, 64)
        c.cache.block_table[int(c.rows[1]), 1] = bad
        st.zero_()
        out = torch.full((2, 4, 2, 64), 7.0, dtype=BF16)
        got = c.call(sd, out=out.cuda(), status=st)
        assert int(st) == sd.S_LEN_RANGE
        k, v = c.old[1]
        keep = [*range(16), *range(32, 40)]
        c.old[1] = (k[:, keep], v[:, keep])
        want, tol = c.want(out)
        assert bool(((got.cpu().double() - want).abs() <= tol).all())
    # a tree with a parent that does not come first: that node is none
    c = Case(sd, 41, BF16, "paged", [20, 40], 4, 1, 2, 64)
    c.parent[0] = [-1, 0, 3, 1]
    st.zero_()
    got = c.call(sd, out=out.cuda(), status=st)
    want, tol = c.want(out)
    assert int(st) == sd.S_TREE and bool(((got.cpu().double() - want).abs() <= tol).all())


def test_attention_refusals(sd):
    c = Case(sd, 47, BF16, "paged", [20, 40], 4, 1, 2, 64)
    q = c.q.cuda()
    for call in (lambda: c.call(sd, q=q[:1]), lambda: c.call(sd, q=q.float()), lambda: c.call(sd, q=q[..., :32].contiguous()),
                 lambda: c.call(sd, out=q[:1]), lambda: c.call(sd, q=q.transpose(2, 3)),
                 lambda: c.call(sd, ws=torch.zeros(64, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(sd.SpecDecError):
        c.call(sd, q=q, out=q)
    with pytest.raises(sd.SpecDecError):
        c.call(sd, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(sd.SpecDecError):
        c.call(sd, scale=NAN)
    with pytest.raises(sd.SpecDecError):
        sd.tree_attention_workspace(1, 300, 4, 2, 64)
    assert sd.tree_attention(q[:0], c.cache, 0, c.kv_new[:, :, :0].cuda().contiguous(),
                             torch.zeros((0, 4), dtype=torch.int32, device="cuda")).shape == (0, 4, 2, 64)


def test_attention_cache_past_4_gib(sd):
    """Pages whose byte offsets pass 2^32 in K and in V (each layer half holds 6.4 GB)."""
    H, page, Dh, n_pages = 8, 16, 128, 196608
    say("cache past 4 GiB", n_pages * H * page * Dh * 2)
    c = Case(sd, 53, BF16, "paged", [100, 37], 6, H, 2, Dh, page, L=1, layer=0)
    small, table = c.cache.pages, c.cache.block_table
    pages = torch.empty((1, 2, n_pages, H, page, Dh), dtype=BF16, device="cuda")
    far = n_pages - 1 - 12345 * torch.arange(small.shape[2], device="cuda") % (n_pages // 4)  # all past 4 GiB
    pages[:, :, far] = small
    table = torch.where(table >= 0, far[table.clamp(min=0).long()].int(), table).contiguous()
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.cache = sd.PagedKV(pages, table, torch.zeros(n_pages, dtype=torch.int32, device="cuda"), z, c.cache.tokens, c.cache.len)
    c.check(sd)


def test_attention_streams(sd):
    """Two calls at once on two streams, each with its own workspace."""
    cases = [Case(sd, 59, BF16, "paged", [3000, 100], 6, 2, 4, 128, L=1, layer=0),
             Case(sd, 61, F16, "rect", [900, 2000], 17, 1, 2, 64, L=1, layer=0)]
    want = [c.check(sd) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            got.append([c.call(sd, out=torch.full_like(w, 7.0)) for w in want[len(got):len(got) + 1] for _ in range(4)])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for x in g:
            assert torch.equal(x, w)


# Query rows per KV head on both sides of every change of tiling, with a row long
# enough to be split; sizes of heads that fill their tiles and that do not.
@pytest.mark.parametrize("dt,Dh", [(BF16, 128), (F16, 72), (F16, 64), (BF16, 256), (F32, 64), (F32, 100), (F32, 200)])
def test_attention_every_tiling(sd, dt, Dh):
    for k, (N, G) in enumerate([(16, 1), (17, 1), (8, 4), (33, 1), (16, 4), (13, 5), (24, 4), (97, 1), (32, 4), (43, 3),
                                (48, 4), (193, 1), (64, 4), (51, 7)]):
        store, page = [("paged", 16), ("rect", 0), ("paged", 1), ("pool", 0), ("paged", 5), ("group", 0)][k % 6]
        say("tiling", dt, Dh, N, G, store, page)
        Case(sd, 400 + k, dt, store, [2531, 1, 0, 130], N, 1, G, Dh, page, L=1, layer=0, used=[N, max(1, N - 5), 1, N],
             wide=k % 2 == 0).check(sd)


def test_attention_shared_keys_pages_past_the_window(sd):
    """More blocks of a row than a workgroup looks up at once."""
    for dt, N, G, page in ((BF16, 40, 1, 1), (F16, 24, 4, 1), (BF16, 100, 1, 2)):
        say("past the window", dt, N, G, page)
        Case(sd, 71, dt, "paged", [5003, 1025, 1024, 1023], N, 1, G, 64, page, L=1, layer=0).check(sd)
    # few segments beside many, so that parts are longer than the window
    say("whole long rows")
    Case(sd, 72, BF16, "paged", [1400] * 8, 40, 40, 1, 64, 1, L=1, layer=0, used=[3] * 8).check(sd)


@pytest.mark.parametrize("dt,N,G", [(BF16, 40, 1), (F16, 24, 4), (BF16, 100, 1), (BF16, 64, 4), (F32, 70, 1)])
def test_attention_shared_keys_bad_pages(sd, dt, N, G):
    """Bad pages under keys that waves share: their positions take no part, in whichever tile they lie."""
    for at in ((1,), (0, 2, 3), (5, 9, 30)):
        for bad in (-1, 1 << 30):
            c = Case(sd, 73, dt, "paged", [20, 500], N, 1, G, 64, 16, L=1, layer=0)
            keep = torch.ones(500, dtype=torch.bool)
            for k in at:
                c.cache.block_table[int(c.rows[1]), k] = bad
                keep[k * 16:k * 16 + 16] = False
            say("bad pages", dt, N, G, at, bad)
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = torch.full((2, N, G, 64), 7.0, dtype=dt)
            got = c.call(sd, out=out.cuda(), status=st)
            assert int(st) == sd.S_LEN_RANGE
            k, v = c.old[1]
            c.old[1] = (k[:, keep], v[:, keep])
            want, tol = c.want(out)
            assert bool(((got.cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dt,N,G", [(BF16, 40, 2), (F16, 96, 1), (BF16, 65, 4), (F32, 50, 1)])
def test_attention_split_rows_with_values_that_are_not_finite(sd, dt, N, G):
    """The last part of a split row holds the tree: its branch that overflowed, and nodes that are not used."""
    c = Case(sd, 79, dt, "paged", [6000], N, 1, G, 64, 16, L=1, layer=0, used=[N - 3])
    parent = np.full(N, -1, np.int32)
    parent[1:N - 3] = [0, 0] + [i - 2 for i in range(3, N - 3)]
    c.parent[:] = parent
    c.kv_new[0, 1, 0, 0, 9, 3] = -float("inf")
    out = torch.full((1, N, G, 64), 7.0, dtype=dt)
    got = c.call(sd, out=out.cuda()).cpu()
    c.kv_new[0, 1, 0, 0, 9, 3] = 0.0
    want, tol = c.want(out)
    lines = T.lines(parent)
    hit = torch.tensor([9 in line for line in lines])
    assert bool((got[0, hit][:, :, 3] == -float("inf")).all())
    got[0, hit, :, 3] = 0.0
    want[0, hit, :, 3] = 0.0
    assert bool(((got.double() - want).abs() <= tol).all())


def test_attention_many_rows(sd):
    """Rows past one wave's lanes, up to the most: none, some and all of them split."""
    rng = np.random.default_rng(5)
    for B, N, G, lens in ((65, 3, 2, [900] * 65), (130, 5, 1, [int(x) for x in rng.integers(0, 200, 130)]),
                          (1024, 1, 1, [int(x) for x in rng.integers(0, 9, 1024)]),
                          (129, 34, 1, [3000, *[1] * 127, 5000]), (200, 2, 1, [*[0] * 199, 30000])):
        say("many rows", B, N, G)
        Case(sd, 83, BF16, "paged", lens, N, 1, G, 64, 16, L=1, layer=0, used=[1 + b % N for b in range(B)]).check(sd)


def test_attention_types_in_turn_on_one_workspace(sd):
    """Types that split the same rows in different ways take turns on one workspace."""
    for N, G, Dh in ((20, 1, 128), (40, 1, 256), (12, 2, 128)):
        ws = sd.tree_attention_workspace(3, N, 2 * G, 2, Dh)
        cases = [Case(sd, 89, dt, "paged", [7000, 5, 2000], N, 2, G, Dh, 16, L=1, layer=0) for dt in (BF16, F32, F16)]
        want = [c.check(sd) for c in cases]
        for k in (1, 0, 1, 2, 1, 1, 0, 2):
            say("types in turn", N, G, Dh, k)
            assert torch.equal(cases[k].check(sd, ws=ws), want[k])


def test_attention_scale_of_zero(sd):
    """Every weight alike: the mean of the values."""
    for N in (6, 40):
        Case(sd, 97, BF16, "rect", [300, 64], N, 2, 2, 64, L=1, layer=0).check(sd, scale=0.0)


@pytest.mark.parametrize("N,G,Dh", [(6, 2, 128), (40, 1, 64)])
def test_attention_graph_follows_the_lengths(sd, N, G, Dh):
    """A captured call plans anew from the lengths of each replay: split, whole, and refused."""
    c = Case(sd, 101, BF16, "paged", [6000, 100], N, 1, G, Dh, 16, L=1, layer=0)
    ws = sd.tree_attention_workspace(2, N, G, 1, Dh)
    q, new, parent, rows = c.q.cuda(), c.kv_new.cuda(), dev(c.parent), dev(c.rows)
    out = torch.full_like(q, 7.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        sd.tree_attention(q, c.cache, 0, new, parent, rows=rows, ws=ws, out=out, status=st)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    old, at = list(c.old), [int(r) for r in c.rows]
    for lens in ((6000, 100), (0, 100), (31, 0), (5000, 99), (-1, 5), (6000, 100)):
        say("replay", lens)
        for r, n in zip(at, lens):
            c.cache.len[r] = n
        out.fill_(7.0)
        st.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = out.cpu()
        if min(lens) < 0:
            assert int(st) == sd.S_LEN_RANGE and bool((got == 7.0).all())
            continue
        assert int(st) == 0
        c.old = [(k[:, :n], v[:, :n]) for (k, v), n in zip(old, lens)]
        want, tol = c.want(torch.full_like(got, 7.0))
        assert bool(((got.double() - want).abs() <= tol).all())
        call()
        assert torch.equal(out.cpu(), got)


# ------------------------------------------------------------ a round, together

def _round(sd, s, ws, keep):
    """One layer-by-layer round of a small model over a paged cache: positions, rotary queries and keys, attention, greedy
    verification, compaction, append.  `keep` holds every output, written in place."""
    sd.tree_positions(s["parent"], s["cache"].len, pos=keep["pos"], status=s["status"])
    for l in range(s["L"]):
        x = keep["qkv"][l]
        x.copy_(s["qkv"][l])
        H, Hq = s["H"], s["Hq"]
        sd.rope(x[:, :, :Hq + H], keep["pos"], s["freq"], out=x[:, :, :Hq + H])
        s["kv_new"][l, 0].copy_(x[:, :, Hq:Hq + H].transpose(1, 2))
        s["kv_new"][l, 1].copy_(x[:, :, Hq + H:].transpose(1, 2))
        sd.tree_attention(x[:, :, :Hq], s["cache"], l, s["kv_new"], s["parent"], out=keep["out"][l], ws=ws["attn"], status=s["status"])
    sd.verify_tree_greedy(s["logits"], s["draft"], s["parent"], s["depth"], ws=ws["greedy"], status=s["status"],
                          accept_len=keep["acc"], next_token=keep["nxt"], path=keep["path"])
    sd.tree_compact(s["kv_new"], s["draft"], keep["path"], keep["acc"], kv_path=keep["kv_path"], draft_path=keep["draft_path"],
                    status=s["status"])
    sd.paged_append(s["cache"], keep["kv_path"], keep["draft_path"], keep["acc"], keep["nxt"], status=s["status"])


def _round_state(sd, seed, dt=BF16, B=5, N=19, L=2, H=2, G=4, Dh=64, V=503, depth=4, page=8):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    Hq = H * G
    lens = rng.integers(0, 120, B).astype(np.int32)
    mb = -(-(int(lens.max()) + 20 * (depth + 1)) // page)
    cache = sd.PagedKV.empty(L, B, H, Dh, B * mb, page, mb, dt)
    cap = int(lens.max()) + 1
    rect = sd.SeqBuf.empty(L, B, H, cap, Dh, dt)
    rect.kv.copy_(torch.randn(rect.kv.shape, generator=g, device="cuda"))
    rect.len.copy_(dev(lens))
    rect.width.fill_(int(lens.max()))
    sd.paged_admit(cache, rect)
    parent = np.stack([T.random_tree(rng, N, int(rng.integers(1, N + 1))) for _ in range(B)])
    logits = torch.randn(B, N, V, generator=g, device="cuda")
    draft = torch.randint(V, (B, N), generator=g, device="cuda", dtype=torch.int32)
    likely = logits.argmax(-1).int().gather(1, dev(np.maximum(parent, 0)).long())
    draft = torch.where(torch.rand(B, N, generator=g, device="cuda") < 0.7, likely, draft)
    s = dict(parent=dev(parent), cache=cache, L=L, H=H, Hq=Hq, depth=depth, logits=logits, draft=draft.contiguous(),
             qkv=torch.randn(L, B, N, Hq + 2 * H, Dh, generator=g, device="cuda").to(dt), freq=sd.rope_frequencies(Dh)[0],
             kv_new=torch.zeros(L, 2, B, H, N, Dh, dtype=dt, device="cuda"), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    keep = dict(pos=torch.zeros(B, N, dtype=torch.int32, device="cuda"), qkv=torch.zeros_like(s["qkv"]),
                out=torch.zeros(L, B, N, Hq, Dh, dtype=dt, device="cuda"), acc=torch.zeros(B, dtype=torch.int32, device="cuda"),
                nxt=torch.zeros(B, dtype=torch.int32, device="cuda"),
                path=torch.zeros(B, depth + 1, dtype=torch.int32, device="cuda"),
                kv_path=torch.zeros(L, 2, B, H, depth + 1, Dh, dtype=dt, device="cuda"),
                draft_path=torch.zeros(B, depth, dtype=torch.int32, device="cuda"))
    ws = dict(attn=sd.tree_attention_workspace(B, N, Hq, H, Dh), greedy=sd.workspace(B, N - 1))
    return s, keep, ws


@pytest.mark.parametrize("seed", range(3))
def test_round_together(sd, seed):
    """Each operator's output against the plain implementation on the outputs before it; the cache after the append holds the
    accepted path's entries and tokens in order."""
    s, keep, ws = _round_state(sd, 70 + seed)
    cache, L, H, Hq = s["cache"], s["L"], s["H"], s["Hq"]
    lens = cache.len.cpu().numpy().copy()
    before = [[[t[:, :lens[b]].clone() for t in _row(cache, l, b)] for b in range(len(lens))] for l in range(L)]
    _round(sd, s, ws, keep)
    torch.cuda.synchronize()
    assert int(s["status"]) == 0
    parent = s["parent"].cpu().numpy()
    pos = T.positions(parent, lens)
    assert np.array_equal(keep["pos"].cpu().numpy(), pos)
    for l in range(L):
        x = s["qkv"][l].cpu()
        want, tol = T.rope(x[:, :, :Hq + H], torch.from_numpy(pos), s["freq"].cpu(), False, 1.0, x[:, :, :Hq + H])
        got = keep["qkv"][l].cpu()
        assert bool(((got[:, :, :Hq + H].double() - want).abs() <= tol).all())
        new = torch.stack([got[:, :, Hq:Hq + H].transpose(1, 2), got[:, :, Hq + H:].transpose(1, 2)])
        want, tol = T.attention(got[:, :, :Hq], before[l], new, parent, 64 ** -0.5, torch.zeros_like(keep["out"][l]).cpu())
        assert bool(((keep["out"][l].cpu().double() - want).abs() <= tol).all())
    target = s["logits"].cpu().numpy().argmax(-1).astype(np.int32)
    draft = s["draft"].cpu().numpy()
    acc, nxt, path = T.greedy(target, draft, parent, s["depth"])
    for k, w in (("acc", acc), ("nxt", nxt), ("path", path)):
        assert np.array_equal(keep[k].cpu().numpy(), w)
    assert acc.max() > 0
    for b in range(len(lens)):
        n = lens[b] + acc[b] + 1
        assert int(cache.len[b]) == n
        tok = [draft[b, i] for i in path[b, 1:acc[b] + 1]] + [nxt[b]]
        assert cache.tokens[b, lens[b]:n].tolist() == tok
        for l in range(L):
            for j, t in enumerate(_row(cache, l, b)):
                assert torch.equal(t[:, :lens[b]], before[l][b][j])
                assert torch.equal(t[:, lens[b]:n], s["kv_new"][l, j, b][:, path[b, :acc[b] + 1]].cpu())


def _row(cache, l, b):
    """K and V [H, positions, Dh] of row b, on the CPU (positions past its length hold anything)."""
    blocks = cache.block_table[b].clamp(min=0).long()
    kv = cache.pages[l][:, blocks].cpu()  # [2, blocks, H, page, Dh]
    return [kv[j].transpose(0, 1).reshape(kv.shape[2], -1, kv.shape[4]) for j in (0, 1)]


def test_round_graph_replays(sd):
    """Three rounds captured in one graph: every replay, with eager work and synchronisation between, gives the eager bytes;
    a second graph shares the workspaces."""
    s, keep, ws = _round_state(sd, 90)
    cache = s["cache"]
    names = ("pages", "block_table", "free_pages", "n_free", "tokens", "len", "sync")
    first = {k: getattr(cache, k).clone() for k in names}

    def reset():
        for k in names:
            getattr(cache, k).copy_(first[k])
        for t in keep.values():
            t.zero_()
        torch.cuda.synchronize()

    def rounds():
        for _ in range(3):
            _round(sd, s, ws, keep)

    def state():
        torch.cuda.synchronize()
        return [t.clone() for t in keep.values()] + [getattr(cache, k).clone() for k in names]

    reset()
    rounds()
    want = state()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            rounds()
        graphs.append(g)
    for rep in range(4):
        reset()
        graphs[rep % 2].replay()
        for x, y in zip(state(), want):
            assert torch.equal(x.view(torch.uint8) if x.dim() else x, y.view(torch.uint8) if y.dim() else y), rep
    assert int(s["status"]) == 0


def test_tree_then_rectangle_realignment(sd):
    """The compacted path goes through the rectangle's realignment, in place and out of place, as a chain's entries do."""
    B, N, H, Dh, depth, L = 4, 12, 2, 64, 5, 2
    rng = np.random.default_rng(8)
    lens = np.array([9, 30, 0, 17], np.int32)
    S = 30
    src = sd.SeqBuf.empty(L, B, H, 64, Dh, F16)
    src.kv.zero_()
    for b in range(B):
        src.kv[:, :, b, :, S - lens[b]:S] = torch.randn(L, 2, H, int(lens[b]), Dh, device="cuda").half()
        src.tokens[b, S - lens[b]:S] = 5
        src.pos[b, S - lens[b]:S] = torch.arange(int(lens[b]), device="cuda", dtype=torch.int32)
        src.mask[b, S - lens[b]:S] = 1
    src.len.copy_(dev(lens))
    src.width.fill_(S)
    parent = np.stack([T.random_tree(rng, N) for _ in range(B)])
    p = torch.softmax(torch.randn(B, N, 300, device="cuda") * 4, -1)
    draft = p.argmax(-1).int().gather(1, dev(np.maximum(parent, 0)).long()).contiguous()
    u = torch.rand(2, B, N, device="cuda")
    kv_new = torch.randn(L, 2, B, H, N, Dh, device="cuda").half()
    acc, nxt, path = sd.verify_tree_sample(p, draft, dev(parent), u[0], u[1], depth)
    kv_path, draft_path = sd.tree_compact(kv_new, draft, path, acc)
    dst = sd.SeqBuf.empty(L, B, H, 64, Dh, F16)
    sd.realign_eqspec(src, dst, kv_path, draft_path, acc, nxt)
    before = src.kv.clone()
    sd.realign_eqspec_inplace(src, kv_path, draft_path, acc, nxt)
    W = int(dst.width)
    assert W == int(src.width) and torch.equal(src.kv[..., :W, :], dst.kv[..., :W, :])
    assert torch.equal(src.tokens[:, :W], dst.tokens[:, :W])
    for b in range(B):
        a = int(acc[b])
        nodes = path[b, :a + 1].long()
        assert torch.equal(dst.kv[:, :, b, :, W - a - 1:W], kv_new[:, :, b][..., nodes, :])
        assert torch.equal(dst.kv[:, :, b, :, W - a - 1 - lens[b]:W - a - 1], before[:, :, b, :, S - lens[b]:S])
        assert dst.tokens[b, W - a - 1:W].tolist() == [*draft[b, nodes[1:]].tolist(), int(nxt[b])]
    assert int(acc.max()) > 0
