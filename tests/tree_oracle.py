"""Plain 64-bit implementations of the tree operators (numpy and torch on the
CPU, one row and node at a time), and the bounds on what the kernels may differ
by from them."""
import math

import numpy as np
import torch

# half a step of rounding to the type, relative to the value
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def lines(parent):
    """For each node of one tree: the nodes from the root to it ([] outside the tree)."""
    out = [[0]]
    for i in range(1, len(parent)):
        p = int(parent[i])
        out.append(out[p] + [i] if 0 <= p < i and out[p] else [])
    return out


def random_tree(rng, N, used=None, wide=False):
    """parent [N]: nodes hang on a random earlier one (near the end unless `wide`); -1 past `used`."""
    used = N if used is None else used
    parent = np.full(N, -1, np.int32)
    for i in range(1, used):
        parent[i] = rng.integers(0 if wide else max(0, i - 4), i)
    return parent


def positions(parent, lens):
    out = np.full(parent.shape, -1, np.int32)
    for b in range(parent.shape[0]):
        for i, line in enumerate(lines(parent[b])):
            if line:
                out[b, i] = lens[b] + len(line) - 1
    return out


def greedy(target, draft, parent, depth):
    """(accept_len, next_token, path) from the target's choices [B, N]."""
    B, N = draft.shape
    acc, nxt, path = np.zeros(B, np.int32), np.zeros(B, np.int32), np.full((B, depth + 1), -1, np.int32)
    for b in range(B):
        cur, path[b, 0] = 0, 0
        while acc[b] < depth:
            kids = [i for i in range(cur + 1, N) if parent[b, i] == cur and draft[b, i] == target[b, cur]]
            if not kids:
                break
            cur = kids[0]
            acc[b] += 1
            path[b, acc[b]] = cur
        nxt[b] = target[b, cur]
    return acc, nxt, path


def sample(p, draft, parent, u_accept, u_draw, depth):
    """(accept_len, next_token, path, the draw's distance to the nearest border relative to the mass)."""
    B, N, V = p.shape
    acc, nxt, path = np.zeros(B, np.int32), np.zeros(B, np.int32), np.full((B, depth + 1), -1, np.int32)
    near = np.full(B, np.inf)
    for b in range(B):
        cur, path[b, 0] = 0, 0
        gone = []
        while acc[b] < depth:
            gone, left, found = [], 1.0, None
            for i in range(cur + 1, N):
                x = int(draft[b, i])
                if parent[b, i] != cur or not 0 <= x < V:
                    continue
                px = 0.0 if x in gone else max(float(p[b, cur, x]), 0.0)
                if float(u_accept[b, i]) * left < px:
                    found = i
                    break
                left -= px
                gone.append(x)
            if found is None:
                break
            cur, gone = found, []
            acc[b] += 1
            path[b, acc[b]] = cur
        w = np.maximum(p[b, cur].astype(np.float64), 0.0)
        cut = w.copy()
        cut[gone] = 0.0
        if cut.sum() > 0:
            w = cut
        c = np.cumsum(w)
        if c[-1] > 0:
            t = float(u_draw[b, cur]) * c[-1]
            nxt[b] = int(np.argmax(c > t))
            near[b] = np.abs(c - t).min() / c[-1]
    return acc, nxt, path, near


def rope(x, pos, freq, interleaved, factor, out):
    """(values in 64 bits, bounds) of the rotation of x [B, N, heads, Dh] into a copy of `out`."""
    x64, y = x.double(), out.double().clone()
    tol = torch.zeros_like(y)
    half = freq.numel()
    if interleaved:
        i0, i1 = torch.arange(0, 2 * half, 2), torch.arange(1, 2 * half, 2)
    else:
        i0, i1 = torch.arange(half), torch.arange(half, 2 * half)
    for b in range(x.shape[0]):
        for n in range(x.shape[1]):
            s = int(pos[b, n])
            if s < 0:
                continue
            a = s * freq.double()
            c, d = torch.cos(a) * factor, torch.sin(a) * factor
            x0, x1 = x64[b, n][:, i0], x64[b, n][:, i1]
            y[b, n] = x64[b, n]
            y[b, n][:, i0], y[b, n][:, i1] = x0 * c - x1 * d, x1 * c + x0 * d
            # the reduced turn in fp32 (half a step of at most 1/2: 2^-26 turns), sine and cosine (4 units
            # of 2^-24 each with the factor), two products and a sum; at |angle| the fp64 product's 2^-53 twice
            e = abs(factor) * (2 * math.pi * 2.0 ** -26 + (4 + 3) * 2.0 ** -24 + a.abs() * 2.0 ** -52)
            tol[b, n][:, i0] = tol[b, n][:, i1] = (x0.abs() + x1.abs()) * e
    return y, tol + y.abs() * HALF[x.dtype] + (2.0 ** -25 if x.dtype == torch.float16 else 0.0)


def attention(q, old, kv_new, parent, scale, out):
    """(values, bounds) of tree attention.  q [B, N, Hq, Dh]; old[b] = (K, V) [H, len, Dh] of each row; kv_new
    [2, B, H, N, Dh]; all on the CPU.  Nodes outside the tree keep `out`."""
    dt = q.dtype
    B, N, Hq, Dh = q.shape
    H = kv_new.shape[2]
    G = Hq // H
    y, tol = out.double().clone(), torch.zeros(out.shape, dtype=torch.float64)
    for b in range(B):
        row = lines(parent[b])
        for h in range(H):
            k0, v0 = old[b][0][h].double(), old[b][1][h].double()
            for i in range(N):
                if not row[i]:
                    continue
                k = torch.cat([k0, kv_new[0, b, h, row[i]].double()])
                v = torch.cat([v0, kv_new[1, b, h, row[i]].double()])
                qs = q[b, i, h * G:(h + 1) * G].double()
                s = qs @ k.t() * scale
                w = torch.softmax(s, -1)
                o = w @ v
                y[b, i, h * G:(h + 1) * G] = o
                n = k.shape[0]
                size = w @ v.abs()  # sum of |w v|
                # a score: Dh + 2 roundings of fp32 in sums of |q k|, scaled and taken to base 2; exp2 another 2 units
                ds = (qs.abs() @ k.abs().t()).amax(-1) * abs(scale) * (Dh + 4) * 2.0 ** -24 + 4 * 2.0 ** -24
                # every weight rounded to the type (in the numerator and, once more, in the sum), the sums over keys
                rel = 2 * ds + (2 * HALF[dt] if dt != torch.float32 else 0.0) + 2 * (n + 16) * 2.0 ** -24
                t = size * rel[:, None] + o.abs() * HALF[dt]
                if dt == torch.float16:  # weights below 2^-14 and outputs below it: half a step of 2^-24
                    t = t + n * 2.0 ** -25 * v.abs().amax(0) + 2.0 ** -25
                tol[b, i, h * G:(h + 1) * G] = t
    return y, tol
