"""GPU parity of the tree operators (positions, rotary positions, verification,
compaction) with plain 64-bit implementations, their status bits and what they
leave untouched."""
import numpy as np
import pytest
import torch

from tests import tree_oracle as T
from tests.gpu_util import bytes_equal, from_np_raw, say, to_np_raw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ragged_kv_realignment_amd as m
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def zero_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ positions

@pytest.mark.parametrize("N", [1, 2, 3, 63, 64, 65, 200, 256])
def test_positions(sd, N):
    say("positions", N)
    rng = np.random.default_rng(N)
    B = 7
    parent = np.stack([T.random_tree(rng, N, int(rng.integers(1, N + 1)), wide=b % 2 == 0) for b in range(B)])
    parent[0] = np.arange(N) - 1          # a chain, the deepest tree
    parent[:, 0] = rng.integers(-9, 9, B)  # not read
    pool = rng.integers(0, 100000, 12).astype(np.int32)
    rows = rng.integers(0, 12, B).astype(np.int32)
    st = zero_status()
    got = sd.tree_positions(dev(parent), dev(pool), rows=dev(rows), status=st)
    assert np.array_equal(got.cpu().numpy(), T.positions(parent, pool[rows])) and int(st) == 0
    got = sd.tree_positions(dev(parent), dev(pool[:B]), status=st)
    assert np.array_equal(got.cpu().numpy(), T.positions(parent, pool)) and int(st) == 0


def test_positions_status(sd):
    parent = np.array([[-1, 0, 1, 3, 5], [-1, 0, -2, 2, 1]], np.int32)  # not before the child; below -1
    st = zero_status()
    got = sd.tree_positions(dev(parent), dev(np.array([4, 9], np.int32)), status=st)
    assert got.cpu().tolist() == [[4, 5, 6, -1, -1], [9, 10, -1, -1, 11]]
    assert int(st) == sd.S_TREE
    for lens, rows in (([4, -1], None), ([4, (1 << 30) + 1], None), ([4, 5], [0, 2]), ([4, 5], [-1, 0])):
        st = zero_status()
        pos = torch.full((2, 5), -77, dtype=torch.int32, device="cuda")
        sd.tree_positions(dev(np.zeros((2, 5), np.int32)), dev(np.array(lens, np.int32)), pos=pos, status=st,
                          rows=None if rows is None else dev(np.array(rows, np.int32)))
        assert int(st) & sd.S_LEN_RANGE and bool((pos == -77).all())
    assert sd.tree_positions(torch.zeros((0, 5), dtype=torch.int32, device="cuda"), dev(np.zeros(0, np.int32))).shape == (0, 5)


# ----------------------------------------------------------------------- rope

ROPE = [  # dtype, B, N, heads, Dh, rot, interleaved
    (torch.bfloat16, 2, 5, 3, 128, 128, False), (torch.bfloat16, 2, 5, 3, 128, 128, True), (torch.float16, 1, 1, 1, 64, 32, False),
    (torch.float16, 3, 7, 40, 96, 24, False), (torch.float16, 3, 7, 40, 96, 24, True), (torch.float32, 2, 3, 2, 16, 16, False),
    (torch.float32, 2, 3, 2, 16, 8, True), (torch.float32, 1, 9, 1, 10, 6, False), (torch.bfloat16, 1, 9, 2, 10, 6, True),
    (torch.bfloat16, 4, 33, 1, 2, 2, False), (torch.float16, 1, 2, 5, 1024, 1024, False), (torch.float32, 1, 3, 2, 256, 128, True),
]


@pytest.mark.parametrize("case", range(len(ROPE)))
def test_rope(sd, case):
    dt, B, N, H, Dh, rot, inter = ROPE[case]
    say("rope", ROPE[case])
    rng = np.random.default_rng(50 + case)
    x = torch.from_numpy(rng.standard_normal((B, N, H, Dh)).astype(np.float32)).to(dt)
    pos = torch.from_numpy(rng.integers(0, 1 << 20, (B, N)).astype(np.int32))
    pos[0, 0] = 0
    if N > 2:
        pos[B - 1, N - 2] = -1
    freq, factor = sd.rope_frequencies(rot, device="cpu"), 1.0
    freq, factor = (freq[0], 1.0) if case % 2 else (freq[0], 1.25)
    out = torch.full_like(x, 7.0)
    want, tol = T.rope(x, pos, freq, inter, factor, out)
    got = out.cuda()
    sd.rope(x.cuda(), pos.cuda(), freq.cuda(), interleaved=inter, factor=factor, out=got)
    assert ((got.cpu().double() - want).abs() <= tol).all()
    # in place, heads of a wider projection, rows and nodes far apart
    wide = torch.full((B, N + 2, H + 3, Dh), 3.0, dtype=dt, device="cuda")
    view = wide[:, 1:N + 1, 2:H + 2]
    view.copy_(x)
    sd.rope(view, pos.cuda(), freq.cuda(), interleaved=inter, factor=factor, out=view)
    kept = (pos < 0)[:, :, None, None]
    assert torch.equal(torch.where(kept, x, got.cpu()), view.cpu())
    view.fill_(3.0)
    assert bool((wide == 3.0).all())
    # an unaligned start and odd strides take the narrow accesses
    flat = torch.zeros(B * N * (H * Dh + 1) + 1, dtype=dt, device="cuda")
    odd = torch.as_strided(flat, (B, N, H, Dh), (N * (H * Dh + 1), H * Dh + 1, Dh, 1), 1)
    odd.copy_(x)
    sd.rope(odd, pos.cuda(), freq.cuda(), interleaved=inter, factor=factor, out=odd)
    assert torch.equal(view.copy_(odd).cpu(), torch.where(kept, x, got.cpu()))


def test_rope_turns_back_and_far(sd):
    """Positions near 2^31: the angle's fp64 form holds; negated frequencies turn back."""
    freq, _ = sd.rope_frequencies(64)
    x = torch.randn(1, 4, 2, 64, device="cuda")
    pos = torch.tensor([[2 ** 31 - 1, 2 ** 30, 12345678, 1]], dtype=torch.int32, device="cuda")
    y = sd.rope(x, pos, freq)
    want, tol = T.rope(x.cpu(), pos.cpu(), freq.cpu(), False, 1.0, x.cpu())
    assert ((y.cpu().double() - want).abs() <= tol).all()
    back = sd.rope(y, pos, -freq)
    assert float((back - x).abs().max()) < 8 * 2.0 ** -20  # two rotations of |x| < 8, a dozen units of 2^-24 each


def test_rope_refusals(sd):
    x = torch.zeros(2, 3, 4, 16, device="cuda")
    pos = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    freq, _ = sd.rope_frequencies(16)
    for call in (lambda: sd.rope(x, pos[:1], freq), lambda: sd.rope(x, pos.long(), freq), lambda: sd.rope(x, pos, freq.float()),
                 lambda: sd.rope(x.transpose(2, 3), pos, freq), lambda: sd.rope(x, pos, freq, out=x[:1]),
                 lambda: sd.rope(x, pos, freq, out=x.half()), lambda: sd.rope(x, pos, freq.cpu())):
        with pytest.raises(ValueError):
            call()
    big, _ = sd.rope_frequencies(18)
    with pytest.raises(sd.SpecDecError):
        sd.rope(x, pos, big)
    with pytest.raises(sd.SpecDecError):  # overlapping, not the same
        w = torch.zeros(2, 4, 4, 16, device="cuda")
        sd.rope(w[:, :3], pos, freq, out=w[:, 1:])
    assert sd.rope(x[:0], pos[:0], freq).shape == (0, 3, 4, 16)


# --------------------------------------------------------------------- greedy

GREEDY = [  # dtype, B, N, V, depth, row stride - V
    (torch.float32, 1, 1, 1, 0, 0), (torch.float32, 2, 2, 5, 1, 0), (torch.bfloat16, 3, 24, 4096, 6, 0),
    (torch.float16, 4, 64, 999, 3, 0), (torch.bfloat16, 2, 65, 20001, 255, 7), (torch.float32, 5, 13, 32000, 4, 32),
    (torch.bfloat16, 2, 256, 1001, 100, 0), (torch.float32, 1, 256, 3, 255, 0),
]


@pytest.mark.parametrize("case", range(len(GREEDY)))
def test_tree_greedy(sd, case):
    dt, B, N, V, depth, gap = GREEDY[case]
    say("tree greedy", GREEDY[case])
    rng = np.random.default_rng(70 + case)
    ws = sd.workspace(B, N - 1)
    for rep in range(3):  # the workspace is left cleared
        parent = np.stack([T.random_tree(rng, N, N if b == 0 else int(rng.integers(1, N + 1)), wide=rep == 1) for b in range(B)])
        if rep == 2:
            parent[0] = np.arange(N) - 1
        buf = torch.from_numpy(rng.integers(-3, 4, (B * N, V + gap)).astype(np.float32)).to(dt).cuda()  # ties everywhere
        logits = torch.as_strided(buf, (B, N, V), (N * (V + gap), V + gap, 1))
        target = logits.float().cpu().numpy().argmax(-1).astype(np.int32)
        draft = rng.integers(0, V, (B, N)).astype(np.int32)
        hit = rng.random((B, N)) < 0.8
        par = np.maximum(parent, 0)
        draft[hit] = np.take_along_axis(target, par, 1)[hit]  # several siblings may hold the choice
        st = zero_status()
        tgt = torch.full((B, N), -5, dtype=torch.int32, device="cuda")
        acc, nxt, path = sd.verify_tree_greedy(logits, dev(draft), dev(parent), depth, ws=ws, status=st, target_tok=tgt)
        want = T.greedy(target, draft, parent, depth)
        assert np.array_equal(tgt.cpu().numpy(), target)
        for g, w in zip((acc, nxt, path), want):
            assert np.array_equal(g.cpu().numpy(), w)
        assert int(st) == 0
    assert not bool(ws.any())


def test_tree_greedy_chain_equals_chain(sd):
    rng = np.random.default_rng(5)
    B, D, V = 6, 7, 5000
    logits = torch.from_numpy(rng.standard_normal((B, D + 1, V)).astype(np.float32)).cuda()
    am = logits.argmax(-1).int()
    draft = am[:, :D].clone()
    for b in range(B):
        draft[b, b:] = torch.where(torch.rand(D - b, device="cuda") < 0.5, draft[b, b:], torch.zeros_like(draft[b, b:]))
    acc, nxt = sd.verify_greedy(logits, draft.contiguous())
    parent = torch.arange(-1, D, dtype=torch.int32, device="cuda").repeat(B, 1)
    nodes = torch.cat([torch.zeros(B, 1, dtype=torch.int32, device="cuda"), draft], 1)
    a2, n2, path = sd.verify_tree_greedy(logits, nodes, parent, D)
    assert torch.equal(acc, a2) and torch.equal(nxt, n2)
    at = torch.arange(D + 1, device="cuda")
    assert torch.equal(path, torch.where(at <= acc[:, None], at, -1 * torch.ones_like(at)).int())


def test_tree_greedy_status(sd):
    logits = torch.zeros(2, 4, 10, device="cuda")
    draft = dev(np.array([[99, 0, 0, 0], [-1, 10, 0, -3]], np.int32))
    good = dev(np.array([[-1, 0, 1, 1], [-1, -1, 0, -1]], np.int32))  # the root's token and unused nodes' are not looked at
    st = zero_status()
    acc, nxt, path = sd.verify_tree_greedy(logits, draft, good, 3, status=st)
    assert int(st) == 0 and acc.tolist() == [2, 1] and path.tolist() == [[0, 1, 2, -1], [0, 2, -1, -1]]
    bad = dev(np.array([[-1, 0, 2, 1], [-1, 0, 0, 0]], np.int32))
    acc, nxt, path = sd.verify_tree_greedy(logits, draft, bad, 3, status=st)
    assert int(st) == sd.S_TREE | sd.S_DRAFT_RANGE and path.tolist() == [[0, 1, 3, -1], [0, 2, -1, -1]]
    acc, nxt, path = sd.verify_tree_greedy(logits[:0], draft[:0], bad[:0], 3)
    assert acc.shape == (0,) and path.shape == (0, 4)


# --------------------------------------------------------------------- sample

SAMPLE = [  # B, N, V, depth
    (1, 1, 1, 0), (3, 9, 7, 4), (4, 24, 32000, 8), (2, 64, 33003, 5), (2, 256, 1000, 255), (5, 17, 152064, 3), (3, 40, 4, 10),
    (1, 8, 262144, 4),
]


@pytest.mark.parametrize("case", range(len(SAMPLE)))
def test_tree_sample(sd, case):
    B, N, V, depth = SAMPLE[case]
    say("tree sample", SAMPLE[case])
    rng = np.random.default_rng(90 + case)
    ws = sd.sample_verify_workspace(B, N - 1, V)
    for rep in range(3):
        p = rng.standard_normal((B, N, V)).astype(np.float32) * 3
        p = np.exp(p - p.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        p[rng.random((B, N, V)) < 0.2] = 0.0
        parent = np.stack([T.random_tree(rng, N, N if b == 0 else int(rng.integers(1, N + 1)), wide=rep == 1) for b in range(B)])
        draft = rng.integers(0, V, (B, N)).astype(np.int32)
        best = np.take_along_axis(p.argmax(-1), np.maximum(parent, 0), 1)
        hit = rng.random((B, N)) < 0.6
        draft[hit] = best[hit]  # siblings with one token among them
        ua, ud = rng.random((2, B, N)).astype(np.float32)
        if rep == 2:
            ua[:, ::2], ud[:, ::3] = 0.0, 0.0
        st = zero_status()
        got = sd.verify_tree_sample(dev(p), dev(draft), dev(parent), dev(ua), dev(ud), depth, ws=ws, status=st)
        acc, nxt, path, near = T.sample(p, draft, parent, ua, ud, depth)
        assert np.array_equal(got[0].cpu().numpy(), acc) and np.array_equal(got[2].cpu().numpy(), path)
        # the order of fp64 sums matters within V * 2^-53 of a border only
        sure = (near > V * 2.0 ** -52) | (ud[np.arange(B), path[np.arange(B), acc]] == 0.0)
        assert np.array_equal(got[1].cpu().numpy()[sure], nxt[sure])
        assert sure.all() or rep < 2
        assert not (int(st) & ~sd.S_PROB)


def test_tree_sample_removed_tokens(sd):
    """Every id a refused child but one: the draw has a single answer, in every run and split; and none left falls back to p."""
    N, V = 200, 9001
    rng = np.random.default_rng(3)
    p = np.zeros((1, N, V), np.float32)
    ids = rng.permutation(V)[:N].astype(np.int32)
    p[0, 0, ids] = 1.0 / N
    draft = np.concatenate([[0], ids[1:]])[None].astype(np.int32)
    parent = np.zeros((1, N), np.int32)
    ua = np.full((1, N), 1 - 2.0 ** -24, np.float32)
    for u in (0.0, 0.5, 1 - 2.0 ** -24):
        ud = np.full((1, N), u, np.float32)
        acc, nxt, path = sd.verify_tree_sample(dev(p), dev(draft), dev(parent), dev(ua), dev(ud), 4)
        assert int(acc) == 0 and int(nxt) == ids[0] and path.tolist() == [[0, -1, -1, -1, -1]]
    p[0, 0, ids[0]] = 0.0
    want = T.sample(p, draft, parent, ua, ud, 4)
    got = sd.verify_tree_sample(dev(p), dev(draft), dev(parent), dev(ua), dev(ud), 4)
    assert int(got[0]) == want[0][0] and int(got[1]) == want[1][0]
    # at the depth limit no child is tried, so none is removed
    got = sd.verify_tree_sample(dev(p), dev(draft), dev(parent), dev(ua), dev(np.zeros((1, N), np.float32)), 0)
    assert int(got[0]) == 0 and int(got[1]) == ids[1:].min()


def test_tree_sample_status(sd):
    p = torch.zeros(2, 3, 8, device="cuda")
    p[1, :, 2] = 1.0
    parent = dev(np.array([[-1, 0, 5], [-1, 0, 0]], np.int32))
    draft = dev(np.array([[0, 1, 1], [0, 8, 2]], np.int32))
    u = torch.full((2, 3), 0.5, device="cuda")
    st = zero_status()
    acc, nxt, path = sd.verify_tree_sample(p, draft, parent, u, u, 2, status=st)
    assert int(st) == sd.S_TREE | sd.S_PROB | sd.S_DRAFT_RANGE
    assert acc.tolist() == [0, 1] and nxt.tolist() == [0, 2] and path.tolist() == [[0, -1, -1], [0, 2, -1]]
    # NaN and negative values have no mass
    q = torch.tensor([float("nan"), -3.0, 0.25, -0.0, 0.75, float("nan"), 0.0, -1.0], device="cuda").repeat(1, 2, 1).contiguous()
    for x, want in ((0.0, 2), (0.2, 2), (0.3, 4), (0.99, 4)):
        ud = torch.full((1, 2), x, device="cuda")
        a, n, _ = sd.verify_tree_sample(q, dev(np.array([[0, 0]], np.int32)), dev(np.array([[-1, 0]], np.int32)), ud, ud, 1)
        assert (int(a), int(n)) == (0, want)


# -------------------------------------------------------------------- compact

COMPACT = [  # dtype, L, B, H, N, Dh, depth
    (torch.bfloat16, 3, 4, 2, 24, 128, 6), (torch.float32, 1, 1, 1, 1, 4, 0), (torch.float16, 2, 7, 3, 13, 80, 12),
    (torch.bfloat16, 5, 3, 5, 256, 8, 255), (torch.float32, 2, 9, 1, 30, 1024, 3), (torch.float16, 0, 3, 2, 6, 64, 4),
]


@pytest.mark.parametrize("case", range(len(COMPACT)))
def test_tree_compact(sd, case):
    dt, L, B, H, N, Dh, depth = COMPACT[case]
    say("compact", COMPACT[case])
    rng = np.random.default_rng(110 + case)
    kv = torch.randint(0, 255, (L, 2, B, H, N, Dh * (4 if dt == torch.float32 else 2)), dtype=torch.uint8, device="cuda").view(dt)
    draft = rng.integers(0, 1 << 30, (B, N)).astype(np.int32)
    acc = rng.integers(0, min(depth, N - 1) + 1, B).astype(np.int32)
    acc[0] = min(depth, N - 1)
    path = np.full((B, depth + 1), -1, np.int32)
    for b in range(B):
        path[b, :acc[b] + 1] = np.concatenate([[0], 1 + np.sort(rng.permutation(N - 1)[:acc[b]])])
    kp = torch.full((L, 2, B, H, depth + 1, Dh), 7.0, dtype=dt, device="cuda")
    dp = torch.full((B, depth), -7, dtype=torch.int32, device="cuda")
    want, wd = to_np_raw(kp).copy(), np.full((B, depth), -7, np.int32)
    src = to_np_raw(kv)
    for b in range(B):
        for j in range(acc[b] + 1):
            want[:, :, b, :, j] = src[:, :, b, :, path[b, j]]
            if j:
                wd[b, j - 1] = draft[b, path[b, j]]
    st = zero_status()
    sd.tree_compact(kv, dev(draft), dev(path), dev(acc), kv_path=kp, draft_path=dp, status=st)
    assert bytes_equal(to_np_raw(kp), want) and np.array_equal(dp.cpu().numpy(), wd) and int(st) == 0


def test_tree_compact_bad_path(sd):
    kv = torch.randn(2, 2, 4, 1, 5, 8, device="cuda")
    draft = torch.arange(20, dtype=torch.int32, device="cuda").view(4, 5)
    path = dev(np.array([[0, 1, 5], [0, 2, 4], [0, -1, -1], [0, 1, -9]], np.int32))
    acc = dev(np.array([2, 2, 3, 1], np.int32))
    kp = torch.full((2, 2, 4, 1, 3, 8), 7.0, device="cuda")
    dp = torch.full((4, 2), -7, dtype=torch.int32, device="cuda")
    st = zero_status()
    sd.tree_compact(kv, draft, path, acc, kv_path=kp, draft_path=dp, status=st)
    assert int(st) == sd.S_TREE
    assert dp.tolist() == [[-7, -7], [7, 9], [-7, -7], [16, -7]]
    assert bool((kp[:, :, [0, 2]] == 7.0).all()) and torch.equal(kp[:, :, 1], kv[:, :, 1][..., [0, 2, 4], :])
    assert torch.equal(kp[:, :, 3, :, :2], kv[:, :, 3, :, :2]) and bool((kp[:, :, 3, :, 2] == 7.0).all())
