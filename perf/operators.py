"""The operators of the key-value cache around the verify step, as they are measured.

Four operators, in the order in which a serving step meets them:

- ``append``: RMS norm of each query and key head, rotary positions, and the
  write of the drafted block's keys and values into the pages of one layer;
- ``attend``: attention of the drafted block (a single token, a chain or a
  tree) over the paged cache;
- ``commit``: after the verify, the accepted nodes' keys and values move
  behind the sequence's prefix in every layer, and the sequence's pages are
  fitted to its new length;
- ``fork``: a sequence is continued twice: whole pages are shared, the last
  one is copied in every layer.

``run`` computes them with elementary torch operations where ``own`` is
false, and with the framework's kernels where it is true.
"""
import math

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6
_THETA = 1e6


# ---- cases --------------------------------------------------------------------------

def _attend(name, N, R, tree, lo, hi, S, Hq=32, Hkv=8, D=128, dtype="bf16", heads_first=False):
    return dict(name=name, op="attend", N=N, R=R, tree=tree, lo=lo, hi=hi, S=S, Hq=Hq, Hkv=Hkv,
                D=D, dtype=dtype, heads_first=heads_first)


def _append(name, N, R, tree, lo, hi, S, Hq=32, Hkv=8, D=128, rot=128, interleaved=False,
            dtype="bf16"):
    return dict(name=name, op="append", N=N, R=R, tree=tree, lo=lo, hi=hi, S=S, Hq=Hq, Hkv=Hkv,
                D=D, rot=rot, interleaved=interleaved, dtype=dtype)


def _commit(name, N, M, accepted, lo, hi, S, L, extra, Hkv=8, D=128, dtype="bf16"):
    return dict(name=name, op="commit", N=N, M=M, accepted=accepted, lo=lo, hi=hi, S=S, L=L,
                extra=extra, Hkv=Hkv, D=D, dtype=dtype)


def _fork(name, N, copies, lo, hi, S, L, Hkv=8, D=128, dtype="bf16"):
    return dict(name=name, op="fork", N=N, copies=copies, lo=lo, hi=hi, S=S, L=L, Hkv=Hkv, D=D,
                dtype=dtype)


def listed():
    return [
        # one request, one new token, a short conversation: latency is all that counts
        _attend("attend_one_token", 1, 1, False, 900, 900, 16),
        # the single-stream verify: 8 sequences, a drafted chain of 8 tokens and its root
        _attend("attend_single_stream", 8, 9, False, 250, 4100, 16),
        # the headline verify's batch: 256 sequences of ordinary, ragged lengths
        _attend("attend_large_batch", 256, 9, False, 128, 2048, 16),
        # the tree verify: 64 nodes and the root of 16 sequences
        _attend("attend_tree", 16, 65, True, 1000, 8200, 32),
        # two long documents, one new token each: the cache's length is split
        _attend("attend_long", 2, 1, False, 65000, 131000, 64),
        # a float32 cache with its heads before its slots, one of its sequences empty
        _attend("attend_float32", 4, 5, False, 0, 2500, 8, 16, 2, 64, "f32", True),
        # a small batch far into long contexts: angles of far positions
        _append("append_small_far", 8, 9, False, 100000, 130000, 16),
        # the largest verify batch: 1024 sequences, 17 rows each, part of the head rotated
        _append("append_max_batch", 1024, 17, False, 0, 100, 16, rot=64, interleaved=True),
        # the tree verify's batch: about four accepted nodes of 64, every layer
        _commit("commit_tree", 16, 64, 4, 10, 200, 32, 36, 0),
        # many trees at once, and room for the next block in the same pass
        _commit("commit_large", 64, 64, 8, 0, 60, 16, 36, 65),
        # one prompt sampled four times
        _fork("fork_one_prompt", 1, 3, 391, 391, 16, 36),
        # a whole batch forked once, large pages
        _fork("fork_batch", 64, 1, 0, 127, 64, 36),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _drawn(rng):
    op = rng.choice(("attend", "attend", "append", "commit", "fork"))
    Hkv = rng.choice((1, 2, 4, 8))
    S = rng.choice((5, 8, 12, 16, 32, 64, 128))
    f32 = rng.random() < 0.2
    dtype = "f32" if f32 else "bf16"
    if op == "attend":
        hi = _log(rng, 1, 131000)
        return _attend("", _log(rng, 1, 256), rng.choice((1, 1, _log(rng, 2, 65))),
                       rng.random() < 0.5, int(hi * rng.random()), hi, S,
                       Hkv * rng.choice((1, 2, 3, 4, 5, 7, 8)), Hkv, rng.choice((64, 96, 128, 128)),
                       dtype, rng.random() < 0.5)
    if op == "append":
        D = rng.choice((64, 96, 128, 128))
        rot = rng.choice((D, D, D // 2, 16))
        hi = _log(rng, 1, 131000)
        return _append("", _log(rng, 1, 1024), _log(rng, 1, 65), rng.random() < 0.5,
                       int(hi * rng.random()), hi, S, Hkv * rng.choice((1, 2, 3, 4, 8)), Hkv, D,
                       rot, rng.random() < 0.5, dtype)
    if op == "commit":
        M = _log(rng, 2, 64)
        hi = _log(rng, 1, 200)
        return _commit("", _log(rng, 1, 64), M, rng.randint(0, min(8, M // 2)),
                       int(hi * rng.random()), hi, S, _log(rng, 1, 36), rng.choice((0, M + 1)),
                       Hkv, rng.choice((64, 128)), dtype)
    hi = _log(rng, 1, 400)
    return _fork("", _log(rng, 1, 64), rng.choice((1, 1, 2, 3)), int(hi * rng.random()), hi, S,
                 _log(rng, 1, 36), Hkv, rng.choice((64, 128)), dtype)


def _pool_tokens(c):
    """Slots of the pages that a case's state holds (the prefix pages of append are shared)."""
    S = c["S"]
    if c["op"] == "append":
        return c["N"] * (c["R"] + 2 * S)
    rows = {"attend": c.get("R"), "commit": c.get("M", 0) + 1, "fork": 0}[c["op"]]
    return c["N"] * ((c["lo"] + c["hi"]) // 2 + rows + S) * (1 + c.get("copies", 0))


def draw(rng):
    largest = {op: max((work(c) for c in listed() if c["op"] == op), key=lambda w: w["bytes"])
               for op in ("attend", "append", "commit", "fork")}
    flops = max(work(c)["flops"] for c in listed() if c["op"] == "attend")
    while True:
        c = _drawn(rng)
        w, e = work(c), 4 if c["dtype"] == "f32" else 2
        share = 8 if c["dtype"] == "f32" else 1  # no tensor cores take float32 as it is
        pool = 2 * c.get("L", 1) * _pool_tokens(c) * c["Hkv"] * c["D"] * e
        if w["bytes"] <= largest[c["op"]]["bytes"] and pool < 3e9 and \
                (c["op"] != "attend" or w["flops"] * share <= flops):
            del c["name"]
            return c


# ---- what a case cannot do without -----------------------------------------------------

def _lens(c):
    n = c["N"]
    return [c["hi"] if n == 1 else c["lo"] + (c["hi"] - c["lo"]) * i // (n - 1) for i in range(n)]


def work(case):
    c, e = case, 4 if case["dtype"] == "f32" else 2
    N, S, H, D = c["N"], c["S"], c["Hkv"], c["D"]
    lens = _lens(c)
    token = 2 * H * D * e  # a token's key and value in one layer
    if c["op"] == "attend":
        R, Hq = c["R"], c["Hq"]
        seen = sum(R * n + (R if c["tree"] else R * (R + 1) // 2) for n in lens)
        return {"bytes": sum(n + R for n in lens) * token + 2 * N * R * Hq * D * e,
                "flops": 4 * Hq * D * seen}
    if c["op"] == "append":
        R, Hq = c["R"], c["Hq"]
        return {"bytes": 2 * N * R * (Hq * D * e + token), "flops": 8 * N * R * (Hq + H) * D}
    if c["op"] == "commit":
        pages = sum(-(-(n + c["M"] + 1) // S) for n in lens)
        return {"bytes": 2 * N * c["accepted"] * c["L"] * token + 8 * pages + 8 * N * c["M"],
                "flops": 0}
    pages = sum(-(-n // S) for n in lens)
    return {"bytes": 2 * c["copies"] * c["L"] * token * sum(n % S for n in lens)
            + 8 * pages * (1 + c["copies"]), "flops": 0}


# ---- inputs ------------------------------------------------------------------------------

def _trees(N, M, g, dev):
    """Parents [N, M] of best-first trees: a node hangs on one of the nodes of the first half
    before it, or on the root."""
    k = torch.arange(M, device=dev)
    u = torch.rand(N, M, generator=g, device=dev)
    return (torch.floor(u * (k // 2 + 1)).to(torch.int32) - 1).contiguous()


def _pool(c, L, P, g, dev):
    shape = (L, P, c["Hkv"], c["S"], c["D"]) if c.get("heads_first") else \
        (L, P, c["S"], c["Hkv"], c["D"])
    t = torch.randn(shape, generator=g, device=dev, dtype=_DTYPE[c["dtype"]])
    return t.transpose(2, 3) if c.get("heads_first") else t


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    N, S, H, D, dt = c["N"], c["S"], c["Hkv"], c["D"], _DTYPE[c["dtype"]]
    order = torch.randperm(N, generator=g, device=dev)
    lens = torch.tensor(_lens(c), dtype=torch.int32, device=dev)[order]
    s = {"case": c, "lens": lens}
    if c["op"] in ("attend", "append"):
        R = c["R"]
        held = [-(-(n + R) // S) for n in _lens(c)]
    elif c["op"] == "commit":
        held = [-(-(n + c["M"] + 1) // S) for n in _lens(c)]
    else:
        held = [-(-n // S) for n in _lens(c)]
    counts = torch.tensor(held, dtype=torch.int64, device=dev)[order]
    width = max(max(held), 1)
    if c["op"] == "commit":
        width += -(-(c["extra"] + c["M"] + 1) // S)
    at = torch.arange(width, device=dev)
    live = at < counts[:, None]
    if c["op"] == "append":  # only the block's own pages are touched: the prefix shares page 0
        first = (lens // S).to(torch.int64)
        live &= at >= first[:, None]
    used = int(live.sum())
    spare = max(N * c.get("copies", 0), N * -(-c.get("extra", 0) // S), 1)
    P = used + spare
    pages = torch.randperm(P, generator=g, device=dev).to(torch.int32)
    table = torch.full((N, width), -1, dtype=torch.int32, device=dev)
    table[live] = pages[:used]
    if c["op"] == "append":
        table[at < first[:, None]] = 0
    L = c.get("L", 1)
    s["k_pages"], s["v_pages"] = _pool(c, L, P, g, dev), _pool(c, L, P, g, dev)
    if c["op"] in ("attend", "append"):
        s["k_pages"], s["v_pages"] = s["k_pages"][0], s["v_pages"][0]
        s["table"] = table
        s["parents"] = _trees(N, R - 1, g, dev) if c["tree"] and R > 1 else None
    if c["op"] == "attend":
        s["q"] = 1.5 * torch.randn(N, R, c["Hq"], D, generator=g, device=dev)
        s["q"] = s["q"].to(dt)
    elif c["op"] == "append":
        Hq = c["Hq"]
        s["qkv"] = torch.randn(N, R, Hq + 2 * H, D, generator=g, device=dev).to(dt)
        s["q_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt)
        s["k_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt)
        half = torch.arange(c["rot"] // 2, dtype=torch.float64, device=dev)
        s["inv_freq"] = _THETA ** (-2.0 * half / c["rot"])
    else:
        if c["op"] == "fork":  # the rows behind the sources are empty and take the copies
            rows = N * (1 + c["copies"])
            full = torch.full((rows, width), -1, dtype=torch.int32, device=dev)
            full[:N] = table
            table = full
            s["lens"] = torch.cat([lens, torch.zeros(rows - N, dtype=torch.int32, device=dev)])
            counts = torch.cat([counts, torch.zeros(rows - N, dtype=torch.int64, device=dev)])
            s["src"] = torch.arange(N, dtype=torch.int32, device=dev).repeat(c["copies"])
            s["dst"] = torch.arange(N, rows, dtype=torch.int32, device=dev)
        else:
            # accepted nodes in the order of their depth, all behind the slots they move to, so
            # that a pass done again leaves the same cache
            M, a = c["M"], c["accepted"]
            behind = torch.rand(N, M, generator=g, device=dev)
            behind[:, :a] = -1.0
            pick = behind.topk(max(a, 1), dim=1).indices.sort(dim=1).values[:, :a]
            s["path_nodes"] = torch.full((N, M), -1, dtype=torch.int32, device=dev)
            s["path_nodes"][:, :a] = pick.to(torch.int32)
            s["path_len"] = torch.full((N,), a, dtype=torch.int32, device=dev)
        refs = torch.zeros(P, dtype=torch.int32, device=dev)
        refs[pages[:used].long()] = 1
        free = torch.full((P,), -1, dtype=torch.int32, device=dev)
        free[:spare] = pages[used:]
        s["pages"] = {"table": table, "counts": counts.to(torch.int32), "refs": refs, "free": free,
                      "n_free": torch.tensor([spare], dtype=torch.int32, device=dev)}
    return s


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import rejection_sampling_verify_b200 as psi
    c = s["case"]
    if c["op"] == "attend":
        return psi.attend_block(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                parents=s["parents"]).o
    if c["op"] == "append":
        Hq, H = c["Hq"], c["Hkv"]
        q, k, v = s["qkv"].split((Hq, H, H), dim=2)
        r = psi.cache_append(q, k, v, s["k_pages"], s["v_pages"], s["table"], s["lens"],
                             q_weight=s["q_weight"], k_weight=s["k_weight"], eps=_EPS,
                             inv_freq=s["inv_freq"], interleaved=c["interleaved"],
                             parents=s["parents"])
        return [r.q, s["k_pages"], s["v_pages"]]
    pages = psi.PageState(**s["pages"])
    if c["op"] == "commit":
        lens = psi.cache_commit(s["k_pages"], s["v_pages"], pages.table, s["lens"],
                                s["path_nodes"], s["path_len"]).lens
        p = psi.cache_resize(pages, lens, c["extra"], c["S"]).pages
    else:
        r = psi.cache_fork(s["k_pages"], s["v_pages"], pages, s["lens"], s["src"], s["dst"])
        lens, p = r.lens, r.pages
    return [s["k_pages"], s["v_pages"], lens, p.table, p.counts, p.refs, p.free, p.n_free]


def _run_plain(s):
    return {"attend": _plain_attend, "append": _plain_append, "commit": _plain_commit,
            "fork": _plain_fork}[s["case"]["op"]](s)


def _ancestors(parents, N, R, dev):
    """[N, R, R], one where column's row is the row itself or one of its ancestors: the inverse
    of (identity - parent matrix), whose entries are whole numbers."""
    if parents is None:
        return torch.ones(R, R, device=dev).tril().expand(N, R, R)
    A = torch.eye(R, device=dev).repeat(N, 1, 1)
    k = torch.arange(1, R, device=dev)
    A[torch.arange(N, device=dev)[:, None], k, parents.long() + 1] = -1.0
    eye = torch.eye(R, device=dev).expand(N, R, R)
    return torch.linalg.solve_triangular(A, eye, upper=False, unitriangular=True)


def _plain_attend(s):
    c = s["case"]
    N, R, Hq, D = s["q"].shape
    H, S, dev = c["Hkv"], c["S"], s["q"].device
    G, T = Hq // H, s["table"].shape[1] * S
    at = s["table"].clamp(min=0).long()
    k = s["k_pages"][at].to(torch.float32).reshape(N, T, H, D).permute(0, 2, 3, 1)
    v = s["v_pages"][at].to(torch.float32).reshape(N, T, H, D).permute(0, 2, 1, 3)
    q = s["q"].to(torch.float32).reshape(N, R, H, G, D).permute(0, 2, 1, 3, 4)
    p = torch.matmul(q.reshape(N, H, R * G, D), k).mul_(D ** -0.5).view(N, H, R, G, T)
    back = torch.arange(T, device=dev) - s["lens"][:, None]  # the slot's row in the block
    anc = _ancestors(s["parents"], N, R, dev) > 0.5
    inside = (back >= 0) & (back < R)
    seen = anc.gather(2, back.clamp(0, R - 1)[:, None, :].expand(N, R, T)) & inside[:, None, :]
    seen |= (back < 0)[:, None, :]
    p.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    p.div_(p.sum(-1, keepdim=True))
    o = torch.matmul(p.view(N, H, R * G, T), v).view(N, H, R, G, D)
    return o.permute(0, 2, 1, 3, 4).reshape(N, R, Hq, D).to(s["q"].dtype)


def _plain_append(s):
    c = s["case"]
    Hq, H, S, D, rot = c["Hq"], c["Hkv"], c["S"], c["D"], c["rot"]
    N, R = s["qkv"].shape[:2]
    dev, dt = s["qkv"].device, s["qkv"].dtype
    x = s["qkv"].to(torch.float32)
    w = torch.cat([s["q_weight"].to(torch.float32).expand(Hq, D),
                   s["k_weight"].to(torch.float32).expand(H, D)])
    y = x[:, :, :Hq + H]
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + _EPS) * w
    depth = _ancestors(s["parents"], N, R, dev).sum(-1).to(torch.int64) - 1
    pos = s["lens"].long()[:, None] + depth
    angle = pos.to(torch.float64)[:, :, None, None] * s["inv_freq"]
    cos, sin = angle.cos().to(torch.float32), angle.sin().to(torch.float32)
    z = y.clone()
    if c["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z[..., 0:rot:2], z[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z[..., :rot // 2], z[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    slot = s["lens"].long()[:, None] + torch.arange(R, device=dev)
    page = s["table"].long().gather(1, slot // S)
    z = z.to(dt)
    s["k_pages"][page, slot % S] = z[:, :, Hq:]
    s["v_pages"][page, slot % S] = s["qkv"][:, :, Hq + H:]
    return [z[:, :, :Hq].contiguous(), s["k_pages"], s["v_pages"]]


def _plain_commit(s):
    c, p = s["case"], s["pages"]
    N, M, S, dev = c["N"], c["M"], c["S"], s["lens"].device
    # move: node j of the path to the slot behind the root's and the nodes' before it
    j = torch.arange(M, device=dev)
    n, j = torch.nonzero(j < s["path_len"][:, None], as_tuple=True)
    to = s["lens"].long()[n] + 1 + j
    frm = s["lens"].long()[n] + 1 + s["path_nodes"].long()[n, j]
    tp, fp = p["table"].long()[n, to // S], p["table"].long()[n, frm // S]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[:, tp, to % S] = pool[:, fp, frm % S]
    lens = s["lens"] + 1 + s["path_len"]
    # fit the pages: give back what is over, lowest page first, then take from the list's end
    width = p["table"].shape[1]
    need = (lens.long() + c["extra"] + S - 1) // S
    held = p["counts"].long()
    at = torch.arange(width, device=dev)
    over = (at >= need[:, None]) & (at < held[:, None])
    refs = p["refs"] - torch.bincount(p["table"][over].long(), minlength=p["refs"].shape[0])
    gone = torch.nonzero((p["refs"] > 0) & (refs == 0))[:, 0]
    free, n_free = p["free"].clone(), p["n_free"].long()
    free[n_free + torch.arange(gone.shape[0], device=dev)] = gone.to(torch.int32)
    n_free = n_free + gone.shape[0]
    table = p["table"].masked_fill(over, -1)
    want = (need - held).clamp(min=0)
    fits = (want.cumsum(0) <= n_free) & (need <= width)
    take = (at >= held[:, None]) & (at < need[:, None]) & fits[:, None]
    n_new = take.sum()
    got = free[(n_free - 1 - torch.arange(N * width, device=dev)).clamp(min=0)][:int(n_new)]
    table[take] = got
    refs[got.long()] = 1
    counts = torch.where(fits, need, torch.minimum(need, held))
    return [s["k_pages"], s["v_pages"], lens, table, counts.to(torch.int32),
            refs.to(torch.int32), free, (n_free - n_new).to(torch.int32)]


def _plain_fork(s):
    c, p = s["case"], s["pages"]
    S, dev = c["S"], s["lens"].device
    src, dst = s["src"].long(), s["dst"].long()
    n = s["lens"].long()[src]
    whole, part = n // S, n % S
    width = p["table"].shape[1]
    at = torch.arange(width, device=dev)
    shared = at < whole[:, None]
    table, refs = p["table"].clone(), p["refs"].clone()
    rows = torch.where(shared, p["table"][src], -1)
    refs += torch.bincount(rows[shared].long(), minlength=refs.shape[0]).to(torch.int32)
    k = torch.nonzero(part > 0)[:, 0]
    new = p["free"][p["n_free"].long() - 1 - torch.arange(k.shape[0], device=dev)]
    rows[k, whole[k]] = new
    refs[new.long()] = 1
    table[dst] = rows
    # the partial pages' slots, in every layer
    i, slot = torch.nonzero(torch.arange(S, device=dev) < part[k][:, None], as_tuple=True)
    frm, to = p["table"].long()[src[k], whole[k]][i], new.long()[i]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[:, to, slot] = pool[:, frm, slot]
    counts, lens = p["counts"].clone(), s["lens"].clone()
    counts[dst] = (whole + (part > 0)).to(torch.int32)
    lens[dst] = n.to(torch.int32)
    return [s["k_pages"], s["v_pages"], lens, table, counts, refs, p["free"].clone(),
            p["n_free"] - k.shape[0]]


# ---- the definitions in 64 bits --------------------------------------------------------------

def _chains(parents, R):
    """For each row of one sequence's block: the rows it sees, root first (host lists)."""
    rows = [[0]]
    for k in range(R - 1):
        up = k if parents is None else int(parents[k]) + 1
        rows.append(rows[up] + [k + 1])
    return rows


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "commit": _exact_commit,
            "fork": _exact_fork}[case["op"]](s)


def _slots(s, n, first, count):
    """(pages, slots) of `count` positions of sequence n from `first` on."""
    S = s["case"]["S"]
    table = s["table"] if "table" in s else s["pages"]["table"]
    t = torch.arange(first, first + count, device=table.device)
    return table[n].long()[t // S], t % S


def _exact_attend(s):
    c = s["case"]
    q = s["q"].to(torch.float64)
    N, R, Hq, D = q.shape
    G = Hq // c["Hkv"]
    out = torch.zeros_like(q)
    lens = s["lens"].tolist()
    tree = None if s["parents"] is None else s["parents"].tolist()
    for n in range(N):
        at = _slots(s, n, 0, lens[n] + R)
        k, v = s["k_pages"][at].to(torch.float64), s["v_pages"][at].to(torch.float64)
        mask = torch.zeros(R, lens[n] + R, dtype=torch.bool)
        mask[:, :lens[n]] = True
        for r, rows in enumerate(_chains(None if tree is None else tree[n], R)):
            mask[r, [lens[n] + x for x in rows]] = True
        mask = mask.to(q.device)
        for h in range(c["Hkv"]):
            score = q[n, :, h * G:(h + 1) * G] @ k[:, h].T / math.sqrt(D)
            score = score.masked_fill(~mask[:, None, :], -math.inf)
            weight = torch.softmax(score, -1)
            out[n, :, h * G:(h + 1) * G] = weight @ v[:, h]
    return out


def _exact_append(s):
    c = s["case"]
    Hq, H, rot = c["Hq"], c["Hkv"], c["rot"]
    x = s["qkv"].to(torch.float64)
    N, R = x.shape[:2]
    rms = (x * x).sum(-1, keepdim=True).div(c["D"]).add(_EPS).sqrt()
    y = x / rms
    y[:, :, :Hq] *= s["q_weight"].to(torch.float64)
    y[:, :, Hq:] *= s["k_weight"].to(torch.float64)
    lens = s["lens"].tolist()
    tree = None if s["parents"] is None else s["parents"].tolist()
    pos = torch.tensor([[lens[n] + len(r) - 1 for r in _chains(tree and tree[n], R)]
                        for n in range(N)], dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.ones_like(s["inv_freq"]).expand(N, R, 1, -1).contiguous(),
                       pos[:, :, None, None] * s["inv_freq"])
    if c["interleaved"]:
        z = torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    k, v = s["k_pages"].to(torch.float64), s["v_pages"].to(torch.float64)
    where = [_slots(s, n, lens[n], R) for n in range(N)]
    page, slot = (torch.stack([w[i] for w in where]) for i in (0, 1))
    k[page, slot] = y[:, :, Hq:Hq + H]
    v[page, slot] = x[:, :, Hq + H:]
    return [y[:, :, :Hq], k, v]


def _exact_commit(s):
    k, v = s["k_pages"], s["v_pages"]
    lens, path, steps = (s[x].tolist() for x in ("lens", "path_nodes", "path_len"))
    for n in range(len(lens)):
        for j in range(steps[n]):
            (tp,), (ts,) = (x.tolist() for x in _slots(s, n, lens[n] + 1 + j, 1))
            (fp,), (fs,) = (x.tolist() for x in _slots(s, n, lens[n] + 1 + path[n][j], 1))
            k[:, tp, ts] = k[:, fp, fs]
            v[:, tp, ts] = v[:, fp, fs]
    return [k, v] + [None] * 6


def _exact_fork(s):
    k, v, S = s["k_pages"], s["v_pages"], s["case"]["S"]
    lens, free = s["lens"].tolist(), s["pages"]["free"].tolist()
    top = int(s["pages"]["n_free"])
    for m in s["src"].tolist():
        if lens[m] % S:
            top -= 1
            page = int(s["pages"]["table"][m, lens[m] // S])
            k[:, free[top], :lens[m] % S] = k[:, page, :lens[m] % S]
            v[:, free[top], :lens[m] % S] = v[:, page, :lens[m] % S]
    return [k, v] + [None] * 6
