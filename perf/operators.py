"""The tree-speculation operators as a user's program calls them, and their plain forms.

A row's drafts form a tree of N nodes: node 0 is the root (the position of the
last committed token), parent[b][i] < i, -1 marks a node that is not used.  One
round rotates queries and keys to the nodes' positions, attends to the cache and
each node's ancestors, verifies the tree against the target, and compacts the
accepted path's entries for the realignment.

With `own` false `run` computes the operators by elementary torch operations;
with `own` true it calls the library."""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one sequence, one new token: plain decoding over a short paged cache, all latency
        dict(name="attend one token", op="attend", dtype="bf16", store="paged", page=16, B=1, N=1, n_lo=1, H=8, G=4, Dh=128,
             len_lo=700, len_hi=700),
        # a round of the 8b-gqa workload with a tree of 24 nodes instead of a chain
        dict(name="attend 8b-gqa round", op="attend", dtype="bf16", store="paged", page=16, B=16, N=24, n_lo=17, H=8, G=4, Dh=128,
             len_lo=256, len_hi=2048),
        # the 7b-mha workload: a left-padded rectangle, one query head per KV head, an odd number of nodes
        dict(name="attend 7b-mha rectangle", op="attend", dtype="f16", store="rect", page=0, B=8, N=13, n_lo=13, H=32, G=1, Dh=128,
             len_lo=128, len_hi=1024),
        # two long contexts, few KV heads with many query heads each, a tree of 64 nodes: the most arithmetic
        dict(name="attend long", op="attend", dtype="bf16", store="paged", page=64, B=2, N=64, n_lo=49, H=2, G=16, Dh=128,
             len_lo=40001, len_hi=65537),
        # the 8b-gqa vocabulary, one sequence with a chain of five drafts
        dict(name="greedy chain", op="greedy", dtype="bf16", B=1, N=6, n_lo=6, V=151936, depth=5),
        # the batch of the 8b-gqa workload with a tree of 24 nodes, some rows with fewer
        dict(name="greedy 8b-gqa tree", op="greedy", dtype="bf16", B=16, N=24, n_lo=17, V=151936, depth=6),
        # one sequence, probabilities of the 7b-mha vocabulary
        dict(name="sample one row", op="sample", B=1, N=9, n_lo=9, V=32000, depth=4),
        # the stoch workload's batch with a tree of 24 nodes
        dict(name="sample stoch tree", op="sample", B=32, N=24, n_lo=17, V=32000, depth=8),
        # the 8b-gqa cache's entries of a round (36 layers, 8 heads)
        dict(name="compact 8b-gqa", op="compact", dtype="bf16", B=16, N=24, n_lo=17, L=36, H=8, Dh=128, depth=6),
        # one sequence of the 7b-mha geometry
        dict(name="compact one row", op="compact", dtype="f16", B=1, N=13, n_lo=13, L=32, H=32, Dh=128, depth=4),
        # queries and keys of one layer of an 8b-gqa round (32 + 8 heads), half layout
        dict(name="rope 8b-gqa round", op="rope", dtype="bf16", B=16, N=24, n_lo=17, heads=40, Dh=128, rot=128, interleaved=False,
             len_lo=256, len_hi=2048, stretch=1.0),
        # a quarter of each head rotated, interleaved, positions past a stretched context, many rows
        dict(name="rope long partial", op="rope", dtype="f16", B=64, N=64, n_lo=40, heads=32, Dh=96, rot=24, interleaved=True,
             len_lo=90000, len_hi=131072, stretch=4.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "greedy", "sample", "compact", "rope"])
    N = _log(rng, 1, 64)
    n_lo = rng.randint(max(1, N * 2 // 3), N)
    if op == "attend":
        H, G = rng.choice([(1, 8), (2, 16), (8, 4), (32, 1), (4, 5), (8, 1), (3, 7)])
        B = _log(rng, 1, 32)
        Dh = rng.choice([64, 128, 128, 80, 256])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        hi = _log(rng, 16, max(17, min(60000, 300000 * 128 // (B * H * Dh), 9 * 10**10 // (4 * B * H * G * N * Dh))))
        store = rng.choice(["paged", "paged", "rect"])
        return dict(op=op, dtype=dtype, store=store, page=rng.choice([16, 64, 24, 5]) if store == "paged" else 0, B=B, N=N,
                    n_lo=n_lo, H=H, G=G, Dh=Dh, len_lo=rng.randint(0, hi), len_hi=hi)
    if op == "greedy":
        return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), B=_log(rng, 1, 8), N=N, n_lo=n_lo,
                    V=rng.choice([32000, 50257, 100003, 65536]), depth=rng.randint(1, 8))
    if op == "sample":
        return dict(op=op, B=_log(rng, 1, 24), N=min(N, 24), n_lo=min(n_lo, 24), V=rng.choice([32000, 50257, 20001, 65536]),
                    depth=rng.randint(1, 8))
    if op == "compact":
        L, H = rng.choice([(36, 8), (32, 32), (40, 2), (5, 3)])
        return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), B=_log(rng, 1, 12), N=min(N, 32), n_lo=min(n_lo, 32), L=L, H=H,
                    Dh=rng.choice([64, 128, 80]), depth=rng.randint(1, 8))
    Dh = rng.choice([64, 128, 96, 256])
    hi = _log(rng, 16, 131072)
    return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), B=_log(rng, 1, 48), N=N, n_lo=n_lo, heads=rng.choice([40, 32, 9, 1]),
                Dh=Dh, rot=rng.choice([Dh, Dh // 2, Dh // 4]), interleaved=rng.choice([False, True]), len_lo=rng.randint(0, hi),
                len_hi=hi, stretch=rng.choice([1.0, 1.0, 8.0]))


# ------------------------------------------------------------------ inputs

def _spread(lo, hi, B):
    """B whole numbers evenly from lo to hi: what a batch holds is the case's, its order the seed's."""
    return np.array([hi if B == 1 else lo + (hi - lo) * b // (B - 1) for b in range(B)], np.int64)


def _trees(rng, B, N, n_lo):
    """Trees whose nodes hang on a recent earlier node, in order, and the nodes in use of each row."""
    n = rng.permutation(_spread(n_lo, N, B))
    parent = np.full((B, N), -1, np.int32)
    for b in range(B):
        for i in range(1, n[b]):
            parent[b, i] = rng.integers(max(0, (i - 1) // 2 - 1), i)
    return parent


def prepare(case, seed):
    c, op = case, case["op"]
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, N = c["B"], c["N"]
    tree = _trees(rng, B, N, c["n_lo"])
    s = dict(case=c, parent=torch.from_numpy(tree).cuda())

    def normal(*shape, dtype):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    if op in ("attend", "rope"):
        lens = rng.permutation(_spread(c["len_lo"], c["len_hi"], B))
        s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    if op == "attend":
        dt, H, G, Dh, top = DT[c["dtype"]], c["H"], c["G"], c["Dh"], c["len_hi"]
        # head vectors of a trained model: a few scores stand out of the rest
        s["q"] = normal(B, N, H * G, Dh, dtype=dt) * 1.5
        s["kv_new"] = normal(1, 2, B, H, N, Dh, dtype=dt)
        s["out"] = torch.zeros(B, N, H * G, Dh, dtype=dt, device="cuda")
        if c["store"] == "paged":
            page = c["page"]
            blocks = -(-top // page) + 1
            n_pages = B * blocks + 3
            s["pages"] = normal(1, 2, n_pages, H, page, Dh, dtype=dt)
            table = rng.permutation(n_pages)[: B * blocks].reshape(B, blocks).astype(np.int32)
            used = -(-lens // page)
            table[np.arange(blocks)[None, :] >= used[:, None]] = -1
            s["table"] = torch.from_numpy(table).cuda()
        else:
            s["kv"] = normal(1, 2, B, H, top + 64, Dh, dtype=dt)
            s["width"] = torch.tensor([top], dtype=torch.int32, device="cuda")
    elif op in ("greedy", "sample"):
        V = c["V"]
        par = s["parent"].long().clamp(min=0)
        rows = torch.arange(B, device="cuda")[:, None]
        if op == "greedy":
            s["logits"] = normal(B, N, V, dtype=DT[c["dtype"]]) * 2
            s["target"] = torch.zeros(B, N, dtype=torch.int32, device="cuda")
            likely = s["logits"].argmax(-1)[rows, par]  # the target's own choice at the parent
        else:
            s["p"] = torch.softmax(normal(B, N, V, dtype=torch.float32).mul_(2.5), -1)
            # a draft model near the target: tokens drawn from the target's own distribution
            likely = torch.multinomial(s["p"].view(B * N, V), 1, generator=g).view(B, N)
            likely = torch.where(torch.rand(B, N, generator=g, device="cuda") < 0.6, s["p"].argmax(-1)[rows, par], likely)
            s["u_accept"] = torch.rand(B, N, generator=g, device="cuda")
            s["u_draw"] = torch.rand(B, N, generator=g, device="cuda")
        other = torch.randint(V, (B, N), generator=g, device="cuda")
        hit = torch.rand(B, N, generator=g, device="cuda") < 0.7
        s["draft"] = torch.where(hit, likely, other).int().contiguous()
    elif op == "compact":
        L, H, Dh, depth, dt = c["L"], c["H"], c["Dh"], c["depth"], DT[c["dtype"]]
        s["kv_new"] = normal(L, 2, B, H, N, Dh, dtype=dt)
        s["draft"] = torch.from_numpy(rng.integers(0, 32000, (B, N)).astype(np.int32)).cuda()
        path = np.full((B, depth + 1), -1, np.int32)
        acc = rng.permutation(_spread(0, min(depth, c["n_lo"] - 1), B)).astype(np.int32)
        for b in range(B):
            path[b, : acc[b] + 1] = np.concatenate([[0], 1 + np.sort(rng.permutation(c["n_lo"] - 1)[: acc[b]])])
        s["path"], s["accept_len"] = torch.from_numpy(path).cuda(), torch.from_numpy(acc).cuda()
        s["kv_path"] = torch.zeros(L, 2, B, H, depth + 1, Dh, dtype=dt, device="cuda")
        s["draft_path"] = torch.zeros(B, depth, dtype=torch.int32, device="cuda")
    else:
        s["x"] = normal(B, N, c["heads"], c["Dh"], dtype=DT[c["dtype"]])
        s["out"] = torch.zeros_like(s["x"])
        # radians per position; a longer context by dividing the positions
        k = np.arange(c["rot"] // 2)
        s["freq"] = torch.from_numpy(10000.0 ** (-2.0 * k / c["rot"]) / c["stretch"]).cuda()
    return s


# ------------------------------------------------------------- plain forms

def _ancestors(parent):
    """[B, N, N] truth values: node j is node i or an ancestor of it; rows and columns of unused nodes are false."""
    B, N = parent.shape
    eye = torch.eye(N, device=parent.device)
    at = torch.arange(N, device=parent.device)
    reach = eye + (parent[:, :, None] == at) * (at > 0)[:, None].float()
    for _ in range(max(1, (N - 1).bit_length())):  # paths of 1, 2, 4, ... steps
        reach = ((reach @ reach) > 0).float()
    reach = reach > 0
    return reach & reach[:, :, :1]


def _plain_attend(s):
    c, parent = s["case"], s["parent"]
    B, N, H, G, Dh, top = c["B"], c["N"], c["H"], c["G"], c["Dh"], c["len_hi"]
    at = torch.arange(top, device="cuda")
    lens = s["lens"].long()
    if c["store"] == "paged":
        page = c["page"]
        block = s["table"].long()[:, at // page].clamp(min=0)
        kv = s["pages"][0][:, block, :, at % page]  # the indexed axes come first: [B, top, 2, H, Dh]
        k, v = kv[:, :, 0].transpose(1, 2).float(), kv[:, :, 1].transpose(1, 2).float()
        seen = at < lens[:, None]
    else:
        k, v = s["kv"][0, 0, :, :, :top].float(), s["kv"][0, 1, :, :, :top].float()
        seen = at >= top - lens[:, None]
    anc = _ancestors(parent)
    k = torch.cat([k, s["kv_new"][0, 0].float()], 2)
    v = torch.cat([v, s["kv_new"][0, 1].float()], 2)
    used = anc[:, :, 0]
    mask = torch.cat([seen[:, None, :].expand(B, N, top), anc | ~used[:, :, None]], 2)  # unused rows see all: never kept
    q = s["q"].float().view(B, N, H, G, Dh).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, Dh)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()).view(B, H, G, N, -1) / math.sqrt(Dh)
    score = score.masked_fill(~mask[:, None, None], -math.inf)
    w = torch.exp(score - score.amax(-1, keepdim=True))
    w = (w / w.sum(-1, keepdim=True)).view(B, H, G * N, -1)
    o = torch.matmul(w, v.contiguous()).view(B, H, G, N, Dh).permute(0, 3, 1, 2, 4).reshape(B, N, H * G, Dh)
    return torch.where(used[:, :, None, None], o.to(s["q"].dtype), s["out"])


def _walk(first, N, depth):
    """The path from the root along first [B, N] (the accepted child of each node, N = none), at most `depth` steps."""
    B = first.shape[0]
    cur = torch.zeros(B, 1, dtype=torch.long, device=first.device)
    acc = torch.zeros(B, 1, dtype=torch.long, device=first.device)
    path = [cur]
    go = torch.ones_like(cur, dtype=torch.bool)
    for _ in range(depth):
        nxt = first.gather(1, cur)
        go = go & (nxt < N)
        cur = torch.where(go, nxt, cur)
        acc = acc + go
        path.append(torch.where(go, nxt, torch.full_like(nxt, -1)))
    return cur[:, 0], acc[:, 0].int(), torch.cat(path, 1).int()


def _first_child(ok, par, N):
    """For every node the lowest child with ok, N if it has none."""
    at = torch.arange(N, device=ok.device)
    is_child = ok[:, None, :] & (par[:, None, :] == at[:, None])  # [B, parent, child]
    return torch.where(is_child, at, torch.full_like(at, N)).amin(-1)


def _plain_greedy(s):
    c, N = s["case"], s["case"]["N"]
    par, used = s["parent"].long(), _ancestors(s["parent"])[:, :, 0]
    x = s["logits"]
    best = x.float().amax(-1, keepdim=True)
    ids = torch.arange(c["V"], device="cuda", dtype=torch.int32)
    t = torch.where(x == best, ids, torch.full_like(ids, c["V"])).amin(-1).long()
    ok = used & (torch.arange(N, device="cuda") > 0) & (s["draft"].long() == t.gather(1, par.clamp(min=0)))
    cur, acc, path = _walk(_first_child(ok, par, N), N, c["depth"])
    return acc, t.gather(1, cur[:, None])[:, 0].int(), path, t.int()


def _plain_sample(s):
    c, N, V = s["case"], s["case"]["N"], s["case"]["V"]
    B = c["B"]
    at, rows = torch.arange(N, device="cuda"), torch.arange(B, device="cuda")
    par, used = s["parent"].long(), _ancestors(s["parent"])[:, :, 0]
    child = used & (at > 0)
    x = s["draft"].long()
    px = s["p"][rows[:, None], par.clamp(min=0), x].double()
    earlier = child[:, :, None] & child[:, None, :] & (par[:, :, None] == par[:, None, :]) & (at[None, :] < at[:, None])
    again = (earlier & (x[:, :, None] == x[:, None, :])).any(-1)  # a token that an earlier sibling has counts once
    px = torch.where(again, torch.zeros_like(px), px)
    rem = 1.0 - (earlier * px[:, None, :]).sum(-1)
    ok = child & (s["u_accept"].double() * rem < px)
    cur, acc, path = _walk(_first_child(ok, par, N), N, c["depth"])
    w = s["p"][rows, cur].double()
    gone = child & (par == cur[:, None]) & (acc < c["depth"])[:, None]
    cut = torch.zeros_like(w).scatter_add_(1, x, gone.double())
    w = torch.where(cut > 0, torch.zeros_like(w), w)
    cum = w.cumsum(-1)
    target = s["u_draw"].gather(1, cur[:, None]).double() * cum[:, -1:]
    ids = torch.arange(V, device="cuda")
    nxt = torch.where(cum > target, ids, torch.full_like(ids, V)).amin(-1)
    return acc, nxt.int(), path


def _plain_compact(s):
    c = s["case"]
    at = torch.arange(c["depth"] + 1, device="cuda")
    keep = at <= s["accept_len"][:, None]
    idx = s["path"].long().clamp(min=0)
    rows = torch.arange(c["B"], device="cuda")[:, None]
    kv = s["kv_new"].permute(2, 4, 0, 1, 3, 5)[rows, idx].permute(2, 3, 0, 4, 1, 5)
    kv = torch.where(keep[None, None, :, None, :, None], kv, s["kv_path"])
    return kv.contiguous(), torch.where(keep[:, 1:], s["draft"].gather(1, idx[:, 1:]), s["draft_path"])


def _plain_rope(s):
    c = s["case"]
    anc = _ancestors(s["parent"])
    used = anc[:, :, 0]
    pos = torch.where(used, s["lens"][:, None] + anc.sum(-1).int() - 1, torch.full_like(s["parent"], -1))
    angle = pos.double()[:, :, None] * s["freq"]
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    x, half = s["x"].float(), c["rot"] // 2
    if c["interleaved"]:
        a, b = x[..., 0 : c["rot"] : 2], x[..., 1 : c["rot"] : 2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half : c["rot"]]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    y = torch.cat([turned, x[..., c["rot"]:]], -1).to(s["x"].dtype)
    return pos, torch.where(used[:, :, None, None], y, s["out"])


# --------------------------------------------------------- the library's calls

def _own(s):
    import ragged_kv_realignment_amd as sd

    c, op = s["case"], s["case"]["op"]
    if op == "attend":
        if "cache" not in s:  # the program's cache and workspace, made once
            rows = c["B"]
            if c["store"] == "paged":
                zeros = torch.zeros(1, dtype=torch.int32, device="cuda")
                free = torch.zeros(s["pages"].shape[2], dtype=torch.int32, device="cuda")
                tokens = torch.zeros(rows, s["table"].shape[1] * c["page"], dtype=torch.int32, device="cuda")
                s["cache"] = sd.PagedKV(s["pages"], s["table"], free, zeros, tokens, s["lens"])
            else:
                tokens = torch.zeros(rows, s["kv"].shape[4], dtype=torch.int32, device="cuda")
                s["cache"] = sd.SeqBuf(s["kv"], tokens, s["lens"], width=s["width"])
            s["ws"] = sd.tree_attention_workspace(c["B"], c["N"], c["H"] * c["G"], c["H"], c["Dh"])
        return sd.tree_attention(s["q"], s["cache"], 0, s["kv_new"], s["parent"], out=s["out"], ws=s["ws"])
    if op == "greedy":
        if "ws" not in s:
            s["ws"] = sd.workspace(c["B"], c["N"] - 1)
        return (*sd.verify_tree_greedy(s["logits"], s["draft"], s["parent"], c["depth"], ws=s["ws"], target_tok=s["target"]), s["target"])
    if op == "sample":
        if "ws" not in s:
            s["ws"] = sd.sample_verify_workspace(c["B"], c["N"] - 1, c["V"])
        return sd.verify_tree_sample(s["p"], s["draft"], s["parent"], s["u_accept"], s["u_draw"], c["depth"], ws=s["ws"])
    if op == "compact":
        return sd.tree_compact(s["kv_new"], s["draft"], s["path"], s["accept_len"], kv_path=s["kv_path"], draft_path=s["draft_path"])
    pos = sd.tree_positions(s["parent"], s["lens"])
    return pos, sd.rope(s["x"], pos, s["freq"], interleaved=c["interleaved"], out=s["out"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "attend":
        return _plain_attend(state)
    if op == "greedy":
        return _plain_greedy(state)
    if op == "sample":
        return _plain_sample(state)
    if op == "compact":
        return _plain_compact(state)
    return _plain_rope(state)


# -------------------------------------------------------------- work and exact

def work(case):
    c, op, B, N = case, case["op"], case["B"], case["N"]
    n = _spread(c["n_lo"], N, B)  # nodes in use
    if op == "attend":
        es, H, G, Dh = ES[c["dtype"]], c["H"], c["G"], c["Dh"]
        keys = int(_spread(c["len_lo"], c["len_hi"], B).sum())
        return {"bytes": es * H * Dh * (2 * keys + int(n.sum()) * (2 + 2 * G)),
                "flops": 4.0 * H * G * Dh * float(n.mean()) * (keys + n.sum() / 2)}
    if op == "greedy":
        return {"bytes": float(ES[c["dtype"]] * c["V"] * int(n.sum())), "flops": float(c["V"] * int(n.sum()))}
    if op == "sample":
        return {"bytes": 4.0 * c["V"] * B + 20.0 * int(n.sum()), "flops": 2.0 * c["V"] * B}
    if op == "compact":
        kept = int((_spread(0, min(c["depth"], c["n_lo"] - 1), B) + 1).sum())
        return {"bytes": 2.0 * ES[c["dtype"]] * 2 * c["L"] * c["H"] * c["Dh"] * kept, "flops": 0.0}
    values = int(n.sum()) * c["heads"] * c["Dh"]
    return {"bytes": 2.0 * ES[c["dtype"]] * values, "flops": 3.0 * values * c["rot"] / c["Dh"]}


def exact(case, seed):
    """attend, compact and rope in 64 bits, row by row from the definition; the verifications return whole numbers."""
    c, op = case, case["op"]
    if op in ("greedy", "sample"):
        return None
    s = prepare(case, seed)
    B, N = c["B"], c["N"]
    parent = s["parent"].cpu().tolist()
    lines = []  # per row and node: the nodes from it to the root, or none
    for b in range(B):
        row = [[0]]
        for i in range(1, N):
            p = parent[b][i]
            row.append(row[p] + [i] if 0 <= p < i and row[p] else [])
        lines.append(row)
    if op == "attend":
        lens = s["lens"].cpu().tolist()
        out = s["out"].double()
        for b in range(B):
            n = lens[b]
            if c["store"] == "paged":
                blocks = s["table"][b, : -(-n // c["page"])].long()
                old = [s["pages"][0, j].index_select(0, blocks).transpose(0, 1).reshape(c["H"], -1, c["Dh"])[:, :n].double() for j in (0, 1)]
            else:
                old = [s["kv"][0, j, b, :, c["len_hi"] - n : c["len_hi"]].double() for j in (0, 1)]
            new = [s["kv_new"][0, j, b].double() for j in (0, 1)]
            for i in range(N):
                if not lines[b][i]:
                    continue
                k, v = (torch.cat([old[j], new[j][:, lines[b][i]]], 1) for j in (0, 1))
                q = s["q"][b, i].double().view(c["H"], c["G"], c["Dh"])
                for h in range(c["H"]):
                    w = torch.softmax(q[h] @ k[h].t() / math.sqrt(c["Dh"]), -1)
                    out[b, i, h * c["G"] : (h + 1) * c["G"]] = w @ v[h]
        return out
    if op == "compact":
        kv, path, acc = s["kv_path"].double(), s["path"].cpu().tolist(), s["accept_len"].cpu().tolist()
        for b in range(B):
            for j in range(acc[b] + 1):
                kv[:, :, b, :, j] = s["kv_new"][:, :, b, :, path[b][j]].double()
        return kv, None
    x, out, lens = s["x"].double(), s["out"].double(), s["lens"].cpu().tolist()
    for b in range(B):
        for i in range(N):
            if not lines[b][i]:
                continue
            turn = torch.polar(torch.ones_like(s["freq"]), s["freq"] * (lens[b] + len(lines[b][i]) - 1))
            out[b, i] = x[b, i]
            h = c["rot"] // 2
            even, odd = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["interleaved"] else (slice(0, h), slice(h, c["rot"]))
            y = torch.complex(x[b, i][:, even].contiguous(), x[b, i][:, odd].contiguous()) * turn
            out[b, i][:, even], out[b, i][:, odd] = y.real, y.imag
    return None, out
