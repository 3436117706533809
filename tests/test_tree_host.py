"""The tree operators without a GPU: refusals of the C ABI and the binding, the
frequencies of rotary positions, and the plain implementations' own properties."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import ragged_kv_realignment_amd as sd
from ragged_kv_realignment_amd import specdec as S
from tests import tree_oracle as T

A = 0x100000  # never dereferenced: every call below fails validation on the host


def _st(*v):
    return (C.c_int64 * 3)(*v)


def test_positions_host_errors():
    f = S.lib().specdec_tree_positions
    assert f(A, -1, 4, A * 2, None, 4, A * 3, None, None) == S.E_ARG
    assert f(A, 4, 0, A * 2, None, 4, A * 3, None, None) == S.E_ARG
    assert f(A, 4, 257, A * 2, None, 4, A * 3, None, None) == S.E_ARG
    assert f(A, 1025, 4, A * 2, None, 4, A * 3, None, None) == S.E_ARG
    assert f(None, 4, 4, A * 2, None, 4, A * 3, None, None) == S.E_ARG
    assert f(A, 4, 4, A * 2, None, 4, None, None, None) == S.E_ARG
    assert f(A, 4, 4, A * 2, None, 4, A + 8, None, None) == S.E_ALIAS
    assert f(None, 0, 4, None, None, 0, None, None, None) == S.OK


def test_rope_host_errors():
    f = S.lib().specdec_rope
    a = dict(x=A, xs=_st(512, 128, 64), out=A * 2, os=_st(512, 128, 64), dt=S.BF16, B=2, N=4, H=2, Dh=64, pos=A * 3, fr=A * 4, rot=64,
             il=0, fa=1.0)

    def call(**kw):
        k = dict(a, **kw)
        return f(k["x"], k["xs"], k["out"], k["os"], k["dt"], k["B"], k["N"], k["H"], k["Dh"], k["pos"], k["fr"], k["rot"],
                 k["il"], k["fa"], None)

    assert call(B=-1) == S.E_ARG
    assert call(Dh=1026) == S.E_ARG
    assert call(Dh=63) == S.E_ARG
    assert call(rot=66) == S.E_ARG
    assert call(rot=7) == S.E_ARG
    assert call(rot=0) == S.E_ARG
    assert call(H=0) == S.E_ARG
    assert call(fa=float("nan")) == S.E_ARG
    assert call(dt=9) == S.E_DTYPE
    assert call(x=None) == S.E_ARG
    assert call(x=A + 1) == S.E_ALIGN
    assert call(out=A + 256) == S.E_ALIAS          # shifted by two heads
    assert call(out=A, os=_st(512, 128, 32)) == S.E_ALIAS  # the same place, other strides
    for st in (_st(512, 0, 64), _st(0, 128, 64), _st(512, 128, 0), _st(512, 64, 64), _st(500, 128, 64), _st(512, 128, -63),
               _st(64, 448, 64)):
        assert call(os=st) == S.E_ALIAS            # elements of out at one place
        assert call(x=A * 2, xs=st, os=st) == S.E_ALIAS
    assert call(B=1 << 20, N=1 << 12) == S.E_ARG
    assert call(B=0) == S.OK


def test_verify_tree_host_errors():
    f = S.lib().specdec_verify_tree_greedy
    need = S.lib().specdec_workspace_bytes(2, 3)
    a = dict(l=A, dt=S.BF16, rs=100, B=2, N=4, V=100, dr=A, par=A, de=3, acc=A, nx=A, path=A, ws=A, n=need)

    def call(**kw):
        k = dict(a, **kw)
        return f(k["l"], k["dt"], k["rs"], k["B"], k["N"], k["V"], k["dr"], k["par"], k["de"], k["acc"], k["nx"], k["path"], None,
                 k["ws"], k["n"], None, None)

    for bad in (dict(B=-1), dict(N=0), dict(N=257), dict(V=0), dict(rs=99), dict(de=-1), dict(de=256), dict(l=None), dict(dr=None),
                dict(par=None), dict(path=None), dict(B=1 << 23)):
        assert call(**bad) == S.E_ARG, bad
    assert call(dt=5) == S.E_DTYPE
    assert call(l=A + 1) == S.E_ALIGN
    assert call(ws=None) == S.E_WORKSPACE
    assert call(n=need - 1) == S.E_WORKSPACE
    assert call(ws=A + 4) == S.E_WORKSPACE
    assert call(B=0) == S.OK
    g = S.lib().specdec_verify_tree_sample
    need = S.lib().specdec_verify_sample_workspace_bytes(2, 3, 100)
    ok = dict(p=A, B=2, N=4, V=100, de=3, u=A, ws=A, n=need)

    def call(**kw):
        k = dict(ok, **kw)
        return g(k["p"], k["B"], k["N"], k["V"], A, A, k["u"], A, k["de"], A, A, A, k["ws"], k["n"], None, None)

    for bad in (dict(B=-1), dict(N=0), dict(N=257), dict(V=0), dict(de=256), dict(p=None), dict(u=None)):
        assert call(**bad) == S.E_ARG, bad
    assert call(p=A + 2) == S.E_ALIGN
    assert call(n=need - 1) == S.E_WORKSPACE
    assert call(ws=A + 8) == S.E_WORKSPACE
    assert call(B=0) == S.OK


def test_compact_host_errors():
    f = S.lib().specdec_tree_compact
    a = dict(kv=A, dt=S.BF16, L=2, B=2, H=2, N=4, Dh=64, dr=A * 2, path=A * 3, acc=A * 4, de=3, out=A * 5, dp=A * 6)

    def call(**kw):
        k = dict(a, **kw)
        return f(k["kv"], k["dt"], k["L"], k["B"], k["H"], k["N"], k["Dh"], k["dr"], k["path"], k["acc"], k["de"], k["out"], k["dp"],
                 None, None)

    for bad in (dict(B=-1), dict(B=1025), dict(N=0), dict(N=257), dict(H=0), dict(L=-1), dict(de=256), dict(kv=None), dict(path=None),
                dict(dp=None), dict(L=1 << 28, H=64)):
        assert call(**bad) == S.E_ARG, bad
    assert call(dt=4) == S.E_DTYPE
    assert call(Dh=4) == S.E_ALIGN
    assert call(kv=A + 8) == S.E_ALIGN
    assert call(out=A + 64) == S.E_ALIAS
    assert call(dp=A * 3) == S.E_ALIAS
    assert call(B=0) == S.OK


def _rect(**kw):
    a = dict(kv=A * 64, tokens=None, pos=None, mask=None, len=A, width=A, rows=4, cap=64, layers=2, heads=2, head_dim=64, dtype=S.BF16)
    a.update(kw)
    return S.SeqBufC(*a.values())


def _pages(**kw):
    a = dict(pages=A * 64, table=A, free=A, nf=A, tok=A, len=A, sync=A, rows=4, n_pages=8, page=16, mb=4, layers=2, heads=2, head_dim=64,
             dtype=S.BF16)
    a.update(kw)
    return S.PagedC(*a.values())


@pytest.mark.parametrize("paged", [False, True])
def test_attention_host_errors(paged):
    L = S.lib()
    a = dict(rows=None, group=0, layer=0, q=A * 2, qs=_st(4 * 4 * 64, 4 * 64, 64), Hq=4, kn=A * 3, par=A, B=4, N=4, sc=0.125, out=A * 4,
             os=_st(4 * 4 * 64, 4 * 64, 64), ws=A * 200, n=1 << 30)

    def call(kv=None, **kw):
        k = dict(a, **kw)
        kv = kv or (_pages() if paged else _rect())
        if paged:
            return L.specdec_tree_attention_paged(C.byref(kv), k["rows"], k["layer"], k["q"], k["qs"], k["Hq"], k["kn"], k["par"], k["B"],
                                                  k["N"], k["sc"], k["out"], k["os"], k["ws"], k["n"], None, None)
        return L.specdec_tree_attention(C.byref(kv), k["rows"], k["group"], k["layer"], k["q"], k["qs"], k["Hq"], k["kn"], k["par"],
                                        k["B"], k["N"], k["sc"], k["out"], k["os"], k["ws"], k["n"], None, None)

    for bad in (dict(B=-1), dict(B=5), dict(N=0), dict(N=257), dict(layer=-1), dict(layer=2), dict(Hq=3), dict(Hq=1), dict(Hq=4096),
                dict(sc=float("inf")), dict(q=None), dict(kn=None), dict(par=None), dict(out=None), dict(qs=None)):
        assert call(**bad) == S.E_ARG, bad
    assert call(q=A * 2 + 8) == S.E_ALIGN
    assert call(kn=A * 3 + 8) == S.E_ALIGN
    assert call(qs=_st(4 * 4 * 64 + 4, 4 * 64, 64)) == S.E_ALIGN
    for st in (_st(4 * 4 * 64, 0, 64), _st(4 * 4 * 64, 4 * 64, 0), _st(4 * 4 * 64, 64, 64), _st(64, 4 * 64, 64)):
        assert call(os=st) == S.E_ALIAS            # elements of out at one place
    assert call(out=A * 2 + 1024) == S.E_ALIAS
    assert call(out=A * 64 + 1024) == S.E_ALIAS
    assert call(out=A * 3 + 1024) == S.E_ALIAS
    assert call(ws=None) == S.E_WORKSPACE
    assert call(n=1024) == S.E_WORKSPACE
    assert call(ws=A * 200 + 8) == S.E_WORKSPACE
    assert call(B=0) == S.OK
    big = dict(head_dim=512)
    assert call(_pages(**big) if paged else _rect(**big), qs=_st(8192, 2048, 512), os=_st(8192, 2048, 512)) == S.E_ARG
    bad = dict(dtype=7)
    assert call(_pages(**bad) if paged else _rect(**bad)) == S.E_DTYPE
    bad = dict(head_dim=4)
    assert call(_pages(**bad) if paged else _rect(**bad)) == S.E_ALIGN
    if paged:
        assert call(_pages(n_pages=1 << 27)) == S.E_ARG  # 2^32 rows of a head
    else:
        assert call(rows=A) == S.E_ARG                   # a rectangle's rows are its batch
        assert call(group=-1) == S.E_ARG
        assert call(_rect(cap=1 << 29)) == S.E_ARG


def test_attention_workspace_sizes():
    f = S.lib().specdec_tree_attention_workspace_bytes
    for bad in ((-1, 4, 4, 2, 64), (1, 0, 4, 2, 64), (1, 257, 4, 2, 64), (1, 4, 3, 2, 64), (1, 4, 4, 0, 64), (1, 4, 4, 2, 257),
                (1, 4, 2050, 2, 64)):
        assert f(*bad) == 0, bad
    assert f(1, 24, 32, 8, 128) == f(16, 24, 32, 8, 128) == f(16, 24, 4, 1, 128) > 0


def test_binding_refuses_host_tensors():
    par = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        sd.tree_positions(par, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        sd.rope(torch.zeros(1, 1, 1, 8), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError):
        sd.verify_tree_greedy(torch.zeros(2, 4, 10), par, par, 3)
    with pytest.raises(ValueError):
        sd.verify_tree_sample(torch.zeros(2, 4, 10), par, par, torch.zeros(2, 4), torch.zeros(2, 4), 3)
    with pytest.raises(ValueError):
        sd.tree_compact(torch.zeros(1, 2, 2, 1, 4, 8), par, par, torch.zeros(2, dtype=torch.int32))


def test_rope_frequencies():
    f, a = sd.rope_frequencies(8, base=10000.0, device="cpu")
    assert a == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-15)
    g, _ = sd.rope_frequencies(8, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(g, f / 4, rtol=1e-15)
    # the base grows until the slowest pair is `factor` times slower; the fastest keeps its pace
    g, _ = sd.rope_frequencies(8, scaling="ntk", factor=4.0, device="cpu")
    assert g[0] == 1.0 and abs(float(g[-1] / f[-1]) - 0.25) < 1e-14
    g, a = sd.rope_frequencies(64, scaling="parts", factor=8.0, original=4096, device="cpu")
    f, _ = sd.rope_frequencies(64, device="cpu")
    turns = f * 4096 / (2 * math.pi)
    assert torch.equal(g[turns > 32], f[turns > 32]) and torch.allclose(g[turns < 1], f[turns < 1] / 8, rtol=1e-15)
    mid = (turns < 32) & (turns > 1)
    assert mid.any() and (g[mid] < f[mid]).all() and (g[mid] > f[mid] / 8).all()
    assert abs(a - (0.1 * math.log(8.0) + 1.0)) < 1e-15
    for bad in (dict(rot=7), dict(rot=8, scaling="other"), dict(rot=8, scaling="parts", factor=2.0), dict(rot=8, factor=0.0),
                dict(rot=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            sd.rope_frequencies(device="cpu", **bad)


@pytest.mark.parametrize("tokens", [(0, 1), (2, 2), (1, 3, 0), (0, 1, 2, 3), ()])
def test_sampled_rule_keeps_the_target_distribution(tokens):
    """The plain implementation's rule over a grid of uniforms: the first token that follows the root is distributed as p,
    whatever the children hold (each accepted child's chance, and the draw's, integrated exactly)."""
    p = np.array([0.125, 0.25, 0.5, 0.125], np.float32)
    N, V, K = 1 + len(tokens), 4, 64
    draft = np.zeros((1, N), np.int32)
    draft[0, 1:] = tokens
    parent = np.zeros((1, N), np.int32)
    got = np.zeros(V)
    # chance that child k is taken: its threshold in u; the midpoints of a grid of multiples of 1/K miss no border
    left, refused, chance = 1.0, 1.0, []
    seen = []
    for x in tokens:
        px = 0.0 if x in seen else float(p[x])
        take = px / left if left > 0 else 0.0
        u = np.zeros((1, N), np.float32)
        u[0, 1 + len(chance)] = np.nextafter(np.float32(take), np.float32(0)) if take > 0 else 0.0
        u[0, 1:1 + len(chance)] = 1 - 2.0 ** -24
        a, _, path, _ = T.sample(np.broadcast_to(p, (1, N, V)), draft, parent, u, u, 1)
        if take > 0 and (take < 1 or not seen):
            assert a[0] == 1 and path[0, 1] == 1 + len(chance)
        got[x] += refused * take
        chance.append(take)
        refused *= 1 - take
        left -= px
        seen.append(x)
    if refused > 0:
        u = np.full((1, N), 1 - 2.0 ** -24, np.float32)
        for k in range(K):
            ud = np.full((1, N), (k + 0.5) / K, np.float32)
            a, nxt, _, _ = T.sample(np.broadcast_to(p, (1, N, V)), draft, parent, u, ud, 1)
            assert a[0] == 0
            got[nxt[0]] += refused / K
    assert np.abs(got - p).max() < 2.0 / K if refused > 0 else np.allclose(got, p)


def test_plain_tree_lines():
    parent = np.array([-7, 0, 0, 1, -1, 4, 9, 3, -3], np.int32)
    assert T.lines(parent) == [[0], [0, 1], [0, 2], [0, 1, 3], [], [], [], [0, 1, 3, 7], []]
