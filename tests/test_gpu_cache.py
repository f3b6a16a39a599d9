"""The key-value cache's operators on the GPU against plain float64 forms
(tests/cache_reference.py), at the sizes, masks, strides and page states
where they can go wrong."""
import itertools
import math
import random

import pytest
import torch

import cache_reference as ref
import rejection_sampling_verify_b200 as psi

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _parents(kind, N, R, seed):
    if kind == "chain" or R == 1:
        return None
    rng = random.Random(seed)
    rows = [[rng.randint(max(-1, k - 6), k - 1) for k in range(R - 1)] for _ in range(N)]
    if kind == "bad":
        for row in rows[::2]:
            k = rng.randrange(R - 1)
            row[k] = rng.choice((k, k + 3, -2, 2**31 - 1))
    return torch.tensor(rows, dtype=torch.int32)


def _cache(N, lens, R, H, D, S, dtype, seed, heads_first=False, spare=3, slack=0):
    """Pools full of noise, a table of shuffled pages, entries past the block -1."""
    g = _gen(seed)
    held = [max(0, -(-(max(n, 0) + R) // S)) for n in lens]
    P = sum(held) + spare
    order = torch.randperm(P, generator=g).tolist()
    width = max(max(held), 1) + slack
    table = torch.full((N, width), -1, dtype=torch.int32)
    for n in range(N):
        for i in range(held[n]):
            table[n, i] = order.pop()
    shape = (P, H, S, D) if heads_first else (P, S, H, D)
    pools = [torch.randn(shape, generator=g).to(DT[dtype]) for _ in range(2)]
    if heads_first:
        pools = [p.transpose(1, 2) for p in pools]
    return pools[0], pools[1], table, torch.tensor(lens, dtype=torch.int32)


def _cuda(t):
    return None if t is None else t.cuda() if t.is_contiguous() else \
        t.transpose(1, 2).contiguous().cuda().transpose(1, 2)


def _check_attend(q, k, v, table, lens, parents=None, scale=None, want_status=0):
    r = psi.attend_block(q.cuda(), _cuda(k), _cuda(v), table.cuda(), lens.cuda(),
                         parents=_cuda(parents), scale=scale, want_lse=True)
    torch.cuda.synchronize()
    o, lse, tol = ref.attend(q, k, v, table, lens, parents, scale)
    there = lens >= 0
    err = (r.o.cpu().double() - o).abs()[there]
    worst = (err / tol[there].clamp(min=1e-30)).max()
    assert bool((err <= tol[there]).all()), float(worst)
    got = r.lse.cpu().double()[there]
    want = lse[there]
    assert torch.equal(torch.isinf(got), torch.isinf(want))
    fin = torch.isfinite(want)
    # the score's error bound, at most 2^-12 here, and the sum's
    assert bool(((got - want).abs()[fin] <= 2.0 ** -12 + 1e-6 * want.abs()[fin]).all())
    assert int(r.status.item()) == want_status
    return r


SHAPES = [
    # N, R, Hq, H, D, S, lens
    (1, 1, 4, 1, 128, 16, [0]),
    (1, 1, 32, 8, 128, 16, [1]),
    (3, 1, 8, 2, 64, 16, [0, 127, 300]),
    (4, 9, 8, 2, 128, 16, [0, 5, 128, 411]),
    (2, 17, 4, 4, 128, 8, [119, 247]),
    (2, 65, 8, 2, 128, 32, [63, 200]),
    (3, 5, 7, 1, 64, 5, [0, 3, 260]),
    (2, 3, 15, 3, 96, 12, [1, 150]),
    (2, 2, 4, 2, 256, 3, [10, 70]),
    (2, 4, 2, 1, 8, 1, [0, 33]),
    (1, 256, 2, 1, 64, 64, [130]),
    (1, 33, 40, 1, 128, 128, [500]),
    (5, 6, 6, 3, 40, 7, [2, 90, 64, 31, 32]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["chain", "tree", "bad"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:6])))
def test_attend_shapes_and_masks(shape, kind, dtype):
    N, R, Hq, H, D, S, lens = shape
    seed = 1000 + SHAPES.index(shape)
    k, v, table, lens = _cache(N, lens, R, H, D, S, dtype, seed, heads_first=seed % 2 == 0)
    q = (1.5 * torch.randn(N, R, Hq, D, generator=_gen(seed + 50))).to(DT[dtype])
    parents = _parents(kind, N, R, seed)
    bad = parents is not None and any(
        c is None for n in range(N) for c in ref.chains(parents[n], R))
    _check_attend(q, k, v, table, lens, parents,
                  want_status=psi.PSI_DEV_BAD_PARENT if bad else 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_long_lengths_are_split_and_joined(dtype):
    """One and two sequences over thousands of positions: partial results of
    many ranges, some of them empty for the short sequence."""
    for seed, (N, R, Hq, H, D, S, lens) in enumerate([
            (1, 1, 4, 1, 128, 16, [5000]), (2, 1, 8, 2, 64, 64, [3, 4097]),
            (2, 9, 4, 1, 128, 16, [2047, 0]), (1, 20, 8, 1, 128, 48, [2600])]):
        k, v, table, lens = _cache(N, lens, R, H, D, S, dtype, 70 + seed)
        q = torch.randn(N, R, Hq, D, generator=_gen(seed)).to(DT[dtype])
        _check_attend(q, k, v, table, lens)


@pytest.mark.parametrize("S", [16, 5])
@pytest.mark.parametrize("D", [8, 40, 56, 72, 96, 120])
def test_attend_heads_smaller_than_their_tile(D, S):
    """bf16 heads that do not fill a tile's 64 or 128 elements, in pages that
    are loaded as boxes and as single rows; what lies behind a head's last
    element in memory is NaN and is neither read as keys nor as values."""
    for seed, (N, R, Hq, H, lens) in enumerate([
            (2, 1, 8, 2, [0, 300]), (2, 5, 6, 2, [127, 40]), (1, 33, 8, 2, [200]),
            (2, 1, 4, 1, [4200, 9]), (1, 20, 8, 1, [2600])]):
        g = 300 + 10 * D + seed
        k, v, table, lens = _cache(N, lens, R, H, D, S, "bf16", g, heads_first=seed % 2 == 1)
        q = torch.randn(N, R, Hq, D, generator=_gen(g)).bfloat16()
        parents = _parents("tree", N, R, g)

        def wide(t):  # the same values with 16 elements of NaN behind each head
            w = torch.full((*t.shape[:-1], D + 16), math.nan, dtype=t.dtype, device="cuda")
            w[..., :D] = t.cuda()
            return w[..., :D]

        r = psi.attend_block(wide(q), wide(k), wide(v), table.cuda(), lens.cuda(),
                             parents=_cuda(parents), want_lse=True)
        o, lse, tol = ref.attend(q, k, v, table, lens, parents)
        assert bool(((r.o.cpu().double() - o).abs() <= tol).all())
        assert torch.equal(torch.isfinite(r.lse.cpu()), torch.isfinite(lse))
        assert int(r.status.item()) == 0
        plain = psi.attend_block(q.cuda(), _cuda(k), _cuda(v), table.cuda(), lens.cuda(),
                                 parents=_cuda(parents))
        assert torch.equal(plain.o, r.o)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_scores_far_apart(dtype):
    """Scores that rise by hundreds along the sequence, and fall: the running
    maximum moves in every tile, and the weights of one end vanish."""
    N, R, Hq, H, D, S = 2, 3, 4, 2, 128, 16
    k, v, table, lens = _cache(N, [700, 701], R, H, D, S, dtype, 5)
    for n, up in ((0, 1), (1, -1)):
        for t in range(int(lens[n])):
            k[int(table[n, t // S]), t % S] = torch.full((H, D), up * (t - 350) * 0.06).to(DT[dtype])
    q = torch.ones(N, R, Hq, D).to(DT[dtype])
    _check_attend(q, k, v, table, lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_attend_scale(dtype, scale):
    k, v, table, lens = _cache(2, [40, 200], 4, 2, 64, 16, dtype, 6)
    q = torch.randn(2, 4, 4, 64, generator=_gen(7)).to(DT[dtype])
    _check_attend(q, k, v, table, lens, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [128, 64, 96])
def test_attend_unseen_values_have_no_influence(dtype, D):
    """NaN and infinities in sibling nodes' keys and values, in slots behind
    the block and in pages of nobody do not reach a row that does not see
    them; a row that sees them shows it."""
    N, R, Hq, H, S = 2, 6, 4, 2, 16
    parents = torch.tensor([[-1, -1, 0, 1, 3]] * N, dtype=torch.int32)
    k, v, table, lens = _cache(N, [37, 130], R, H, D, S, dtype, 8)
    q = torch.randn(N, R, Hq, D, generator=_gen(9)).to(DT[dtype])
    clean = _check_attend(q, k, v, table, lens, parents)
    used = set()
    for n in range(N):
        for t in range(int(lens[n]) + R):
            used.add((int(table[n, t // S]), t % S))
    k2, v2 = k.clone(), v.clone()
    for p in range(k.shape[0]):
        for s in range(S):
            if (p, s) not in used:
                k2[p, s], v2[p, s] = math.nan, math.inf
    bad_row = 2  # node 1: seen by itself and nodes 3 and 4 (rows 2, 4, 5)
    for n, (x, y) in enumerate([(math.nan, math.nan), (math.inf, -math.inf)]):
        t = int(lens[n]) + bad_row
        k2[int(table[n, t // S]), t % S, :, 1] = x
        v2[int(table[n, t // S]), t % S, :, 3] = y
    r = psi.attend_block(q.cuda(), k2.cuda(), v2.cuda(), table.cuda(), lens.cuda(),
                         parents=parents.cuda())
    for row in range(R):
        same = torch.equal(r.o[:, row], clean.o[:, row])
        assert same == (row not in (2, 4, 5)), row
    assert not bool(torch.isfinite(r.o[:, 2, :, 3].float()).any())


def test_attend_infinite_values_that_are_seen():
    """A seen value of inf gives inf, as the sum does."""
    for dtype, D in itertools.product(DT, (64, 128)):
        k, v, table, lens = _cache(1, [50], 2, 1, D, 16, dtype, 10)
        v[int(table[0, 1]), 3, 0, 5] = math.inf
        q = torch.randn(1, 2, 2, D, generator=_gen(11)).to(DT[dtype])
        o = psi.attend_block(q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda()).o.float()
        assert bool(torch.isposinf(o[..., 5]).all())
        o[..., 5] = 0
        assert bool(torch.isfinite(o).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_padded_batch_and_bad_pages(dtype):
    """Absent sequences' rows stay as they were; positions without a page are
    left out and flagged; a row left with nothing gives zeros and -inf."""
    N, R, Hq, H, D, S = 5, 2, 4, 2, 128, 16
    k, v, table, lens = _cache(N, [30, -1, 50, 0, -7], R, H, D, S, dtype, 12)
    q = torch.randn(N, R, Hq, D, generator=_gen(13)).to(DT[dtype])
    table[0, 0] = k.shape[0]      # past the pool
    table[2, 1] = -5
    table[3, :] = -1              # nothing at all
    lens[2] = 60                  # past the row's last page
    out = psi.AttendResult(torch.full((N, R, Hq, D), 7.0, dtype=DT[dtype], device="cuda"),
                           torch.full((N, R, Hq), 7.0, device="cuda"),
                           torch.zeros(1, dtype=torch.int32, device="cuda"))
    psi.attend_block(q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda(), out=out)
    o, lse, tol = ref.attend(q, k, v, table, lens)
    for n in (1, 4):
        assert bool((out.o[n] == 7).all()) and bool((out.lse[n] == 7).all())
    for n in (0, 2):
        assert bool(((out.o[n].cpu().double() - o[n]).abs() <= tol[n]).all())
    assert bool((out.o[3] == 0).all()) and bool(torch.isneginf(out.lse[3]).all())
    assert int(out.status.item()) == psi.PSI_DEV_BAD_PAGE


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", [16, 5])
@pytest.mark.parametrize("D", [64, 128, 96])
def test_attend_bad_pages_inside_a_tree_block(D, S, dtype):
    """Positions of the block itself lose their page, in pools whose other
    slots hold NaN and inf: the rows that see them go on without them."""
    N, R, Hq, H = 3, 40, 6, 2
    k, v, table, lens = _cache(N, [100, 7, 250], R, H, D, S, dtype, 21)
    used = torch.zeros(k.shape[:2], dtype=torch.bool)
    for n in range(N):
        for t in range(int(lens[n]) + R):
            used[int(table[n, t // S]), t % S] = True
    k[~used], v[~used] = math.inf, math.nan
    q = torch.randn(N, R, Hq, D, generator=_gen(22)).to(DT[dtype])
    parents = _parents("tree", N, R, 23)
    for n in range(N):
        held = int((table[n] >= 0).sum())
        table[n, held - 2] = -1 if n else k.shape[0] + 3
        table[n, 0] = -7
    _check_attend(q, k, v, table, lens, parents, want_status=psi.PSI_DEV_BAD_PAGE)


def test_attend_lengths_at_and_past_the_table():
    """The table ends before, at and inside the block, and far before it."""
    for dtype in DT:
        k, v, table, lens = _cache(4, [60, 60, 60, 60], 4, 2, 128, 16, dtype, 24)
        q = torch.randn(4, 4, 4, 128, generator=_gen(25)).to(DT[dtype])
        lens = torch.tensor([61, 64, 80, 2**31 - 1], dtype=torch.int32)
        r = psi.attend_block(q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda())
        o, _, tol = ref.attend(q, k, v, table, torch.tensor([61, 64, 64, 64]))
        for n in (0, 1):
            assert bool(((r.o[n].cpu().double() - o[n]).abs() <= tol[n]).all())
        # past the table a row sees all 64 positions that the table holds, and nothing else
        for n in (2, 3):
            assert bool(((r.o[n].cpu().double() - o[n]).abs() <= tol[n]).all())
        assert int(r.status.item()) == psi.PSI_DEV_BAD_PAGE


def test_attend_a_row_of_nan_leaves_the_others():
    """A NaN query gives NaN for its row and head alone; a whole row at -inf
    scores next to finite ones has no weight."""
    for dtype, D in itertools.product(DT, (64, 128)):
        k, v, table, lens = _cache(2, [300, 40], 5, 1, D, 16, dtype, 26)
        q = torch.randn(2, 5, 4, D, generator=_gen(27)).to(DT[dtype])
        clean = psi.attend_block(q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda()).o
        q[1, 2, 3, 7] = math.nan
        o = psi.attend_block(q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda()).o
        assert bool(torch.isnan(o[1, 2, 3]).all())
        o[1, 2, 3] = clean[1, 2, 3]
        assert torch.equal(o, clean)


def test_short_and_long_forms_of_a_call_agree():
    """The compiled binding's calls and those with the caller's own outputs
    give the same bits, on the default and on another stream."""
    N, R, Hq, H, D, S, L, P = 3, 5, 8, 2, 128, 16, 2, 40
    g = _gen(28)
    qkv = torch.randn(N, R, Hq + 2 * H, D, generator=g).bfloat16().cuda()
    q, kk, vv = qkv.split((Hq, H, H), dim=2)
    pages = psi.cache_resize(psi.PageState.empty(N, 8, P),
                             torch.tensor([20, 3, 50], dtype=torch.int32).cuda(), R, S).pages
    lens = torch.tensor([20, 3, 50], dtype=torch.int32).cuda()
    kp, vp = (torch.randn(L, P, S, H, D, generator=g).bfloat16().cuda() for _ in range(2))
    inv, _ = psi.rope_frequencies(D)
    path = torch.tensor([[0, 2, -1, -1], [1, 3, -1, -1], [-1] * 4], dtype=torch.int32).cuda()
    steps = torch.tensor([2, 2, 0], dtype=torch.int32).cuda()
    src, dst = (torch.tensor([x], dtype=torch.int32).cuda() for x in (2, 1))

    def word():
        return torch.zeros(1, dtype=torch.int32, device="cuda")

    def like(s):
        return psi.PageState(*(torch.empty_like(t) for t in (s.table, s.counts, s.refs, s.free,
                                                             s.n_free)))

    def run(given, stream=None):
        k, v = kp.clone(), vp.clone()
        torch.cuda.synchronize()
        a = psi.cache_append(q, kk, vv, k[0], v[0], pages.table, lens, inv_freq=inv, stream=stream,
                             out=psi.AppendResult(torch.empty(N, R, Hq, D, dtype=q.dtype,
                                                              device="cuda"), word())
                             if given else None)
        o = psi.attend_block(a.q, k[0], v[0], pages.table, lens, want_lse=True, stream=stream,
                             out=psi.AttendResult(torch.empty_like(a.q),
                                                  torch.empty(N, R, Hq, device="cuda"), word())
                             if given else None)
        c = psi.cache_commit(k, v, pages.table, lens, path, steps, stream=stream,
                             out=psi.CommitResult(torch.empty_like(lens), word()) if given else None)
        z = psi.cache_resize(pages, c.lens, 0, S, stream=stream,
                             out=psi.ResizeResult(like(pages), word()) if given else None)
        gone = c.lens.clone()
        torch.cuda.synchronize()
        gone[1] = 0
        e = psi.cache_resize(z.pages, gone, 0, S, stream=stream).pages
        f = psi.cache_fork(k, v, e, gone, src, dst, stream=stream,
                           out=psi.ForkResult(like(e), torch.empty_like(gone), word())
                           if given else None)
        torch.cuda.synchronize()
        assert all(int(x.status.item()) == 0 for x in (a, o, c, z, f))
        return [a.q, o.o, o.lse, c.lens, z.pages.table, z.pages.refs, f.pages.table, f.pages.counts,
                f.pages.refs, f.pages.n_free, f.lens, k, v]

    want = run(False)
    for got in (run(True), run(False, torch.cuda.Stream()), run(True, torch.cuda.Stream())):
        for x, y in zip(want, got):
            assert torch.equal(x, y)
    with torch.cuda.stream(torch.cuda.Stream()):
        for x, y in zip(want, run(False)):
            assert torch.equal(x, y)
    with pytest.raises(psi.PsiError):  # what the sizes refuse, refused the same in both forms
        psi.cache_resize(pages, lens, -1, S)
    with pytest.raises(ValueError, match="lens"):
        psi.attend_block(q, kp[0], vp[0], pages.table, lens.long())


def test_attend_repeats_and_does_not_depend_on_the_batch():
    """The same call gives the same bits; a sequence's result is the same in
    another place of a batch of the same shape."""
    for dtype in DT:
        k, v, table, lens = _cache(4, [300, 20, 900, 77], 9, 2, 128, 16, dtype, 14)
        q = torch.randn(4, 9, 8, 128, generator=_gen(15)).to(DT[dtype])
        args = [x.cuda() for x in (q, k, v, table, lens)]
        a, b = psi.attend_block(*args).o, psi.attend_block(*args).o
        assert torch.equal(a, b)
        perm = torch.tensor([2, 0, 3, 1])
        c = psi.attend_block(q[perm].cuda(), args[1], args[2], table[perm].cuda(),
                             lens[perm].cuda()).o
        assert torch.equal(c, a[perm.cuda()])


def test_attend_strided_queries_streams_and_workspace():
    """Queries sliced from one projection, a caller's workspace, another
    stream, and a graph replayed on new inputs."""
    N, R, Hq, H, D, S = 3, 9, 8, 2, 128, 16
    k, v, table, lens = _cache(N, [100, 700, 33], R, H, D, S, "bf16", 16)
    qkv = torch.randn(N, R, Hq + 2 * H, D, generator=_gen(17)).bfloat16().cuda()
    q = qkv[:, :, :Hq]
    kc, vc, tc, lc = k.cuda(), v.cuda(), table.cuda(), lens.cuda()
    plain = psi.attend_block(q.contiguous(), kc, vc, tc, lc).o
    assert torch.equal(psi.attend_block(q, kc, vc, tc, lc).o, plain)
    need = psi.psi_attend_block_workspace_bytes(
        psi.cache._layout(kc, vc, False), N, R, Hq, table.shape[1])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = psi.AttendResult(torch.empty_like(plain), None,
                           torch.zeros(1, dtype=torch.int32, device="cuda"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        psi.attend_block(q, kc, vc, tc, lc, workspace=ws, out=out)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out.o, plain)
    # two graphs that share the workspace, replayed in turn
    other = psi.AttendResult(torch.empty_like(plain), None, out.status)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        psi.attend_block(q, kc, vc, tc, lc, workspace=ws, out=out)
    with torch.cuda.graph(g2):
        psi.attend_block(q, vc, kc, tc, lc, workspace=ws, out=other)
    for i in range(2):
        qkv.copy_(torch.randn(qkv.shape, generator=_gen(18 + i)).bfloat16())
        lc.copy_(torch.tensor([50 + i, 650, 0], dtype=torch.int32))
        out.o.zero_()
        other.o.zero_()
        for g in (g1, g2, g1):
            g.replay()
        assert torch.equal(out.o, psi.attend_block(q, kc, vc, tc, lc).o)
        assert torch.equal(other.o, psi.attend_block(q, vc, kc, tc, lc).o)


def test_attend_offsets_beyond_32_bits():
    """Pages whose element offsets pass 2^32 (a pool of more than 8 GB)."""
    S, H, D = 16, 8, 128
    P = (2**32 // (S * H * D)) + 40
    k = torch.zeros(P, S, H, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(P, S, H, D, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[P - 1, 3, P - 7]], dtype=torch.int32)
    g = _gen(20)
    for p in table[0].tolist():
        k[p] = torch.randn(S, H, D, generator=g).bfloat16()
        v[p] = torch.randn(S, H, D, generator=g).bfloat16()
    lens = torch.tensor([40], dtype=torch.int32)
    q = torch.randn(1, 2, 16, D, generator=g).bfloat16()
    r = psi.attend_block(q.cuda(), k, v, table.cuda(), lens.cuda())
    small = torch.zeros(3, S, H, D, dtype=torch.bfloat16), torch.zeros(3, S, H, D,
                                                                       dtype=torch.bfloat16)
    for i, p in enumerate(table[0].tolist()):
        small[0][i], small[1][i] = k[p].cpu(), v[p].cpu()
    o, _, tol = ref.attend(q, *small, torch.tensor([[0, 1, 2]]), lens)
    assert bool(((r.o.cpu().double() - o).abs() <= tol).all())
    # the write lands there too
    x = torch.randn(1, 2, H, D, generator=g).bfloat16().cuda()
    psi.cache_append(q.cuda(), x, x, k, v, table.cuda(), lens.cuda())
    assert torch.equal(k[P - 7, 8:10], x[0]) and torch.equal(v[P - 7, 8:10], x[0])


# ---- append ------------------------------------------------------------------------

APPENDS = [
    # N, R, Hq, H, D, rot, interleaved, S, lens
    (2, 1, 4, 1, 128, 128, False, 16, [0, 15]),
    (3, 9, 8, 2, 128, 128, False, 16, [0, 7, 130000]),
    (2, 17, 4, 4, 128, 64, True, 8, [100, 3]),
    (2, 5, 7, 1, 64, 64, True, 5, [0, 999999]),
    (2, 6, 6, 3, 96, 48, False, 12, [11, 12]),
    (1, 33, 2, 2, 256, 256, False, 64, [64]),
    (2, 3, 3, 1, 40, 18, False, 1, [0, 5]),
    (2, 3, 3, 1, 40, 2, True, 3, [2, 6]),
    (2, 4, 2, 1, 8, 0, False, 16, [3, 14]),
    (1, 256, 2, 1, 64, 16, False, 1024, [800]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["chain", "tree", "bad"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("case", APPENDS, ids=lambda s: "x".join(map(str, s[:8])))
def test_append(case, norm, kind, dtype):
    N, R, Hq, H, D, rot, inter, S, lens = case
    seed = 300 + APPENDS.index(case)
    k, v, table, lens = _cache(N, [min(n, 200) for n in lens], R, H, D, S, dtype, seed,
                               heads_first=seed % 2 == 1)
    lens_far = torch.tensor(case[8], dtype=torch.int32)
    if not torch.equal(lens, lens_far):  # a far position: its page is all the row needs to hold
        width = -(-(int(lens_far.max()) + R) // S)
        far = torch.full((N, width), -1, dtype=torch.int32)
        own = iter(torch.randperm(k.shape[0], generator=_gen(seed)).tolist())
        for n in range(N):
            for i in range(int(lens_far[n]) // S, -(-(int(lens_far[n]) + R) // S)):
                far[n, i] = next(own)
        table, lens = far, lens_far
    g = _gen(seed + 1)
    qkv = torch.randn(N, R, Hq + 2 * H, D, generator=g).to(DT[dtype])
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).to(DT[dtype]) if norm else None
              for _ in range(2))
    inv, rs = (None, 1.0) if rot == 0 else psi.rope_frequencies(rot, 1e6, 4.0, "yarn",
                                                                device="cpu")
    parents = _parents(kind, N, R, seed)
    kg, vg = _cuda(k), _cuda(v)
    dev = qkv.cuda()
    out = psi.AppendResult(torch.full((N, R, Hq, D), 7.0, dtype=DT[dtype], device="cuda"),
                           torch.zeros(1, dtype=torch.int32, device="cuda"))
    psi.cache_append(dev[:, :, :Hq], dev[:, :, Hq:Hq + H], dev[:, :, Hq + H:], kg, vg,
                     table.cuda(), lens.cuda(), q_weight=_cuda(qw), k_weight=_cuda(kw), eps=1e-5,
                     inv_freq=_cuda(inv), interleaved=inter, rope_scale=rs, parents=_cuda(parents),
                     out=out)
    q, kk, vv, valid, tolq, tolk = ref.append(
        qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:], lens, qw, kw, 1e-5, inv, inter,
        rs, parents)
    assert int(out.status.item()) == (0 if bool(valid.all()) else psi.PSI_DEV_BAD_PARENT)
    got, kc, vc = out.q.cpu(), kg.cpu(), vg.cpu()
    wk, wv = k.double(), v.clone()
    tk = torch.zeros_like(wk)
    for n in range(N):
        for r in range(R):
            t = int(lens[n]) + r
            if valid[n, r]:
                p = int(table[n, t // S])
                wk[p, t % S], wv[p, t % S], tk[p, t % S] = kk[n, r], vv[n, r], tolk[n, r]
    assert bool(((got.double() - q).abs() <= tolq)[valid].all())
    assert bool((got[~valid] == 7).all())
    assert bool(((kc.double() - wk).abs() <= tk).all())  # every other slot as it was
    assert torch.equal(vc, wv)


def test_append_in_place_absent_sequences_and_bad_pages():
    N, R, Hq, H, D, S = 4, 3, 4, 2, 64, 4
    for dtype in DT:
        k, v, table, lens = _cache(N, [6, -1, 2, 9], R, H, D, S, dtype, 40)
        table[2, 0] = -1           # row 0 and 1 of the block lose their slots
        lens[3] = 11               # the last rows lie past the table
        g = _gen(41)
        q0 = torch.randn(N, R, Hq, D, generator=g).to(DT[dtype])
        x, y = (torch.randn(N, R, H, D, generator=g).to(DT[dtype]) for _ in range(2))
        inv, _ = psi.rope_frequencies(D, device="cpu")
        kg, vg, q = k.cuda(), v.cuda(), q0.cuda()
        out = psi.AppendResult(q, torch.zeros(1, dtype=torch.int32, device="cuda"))
        psi.cache_append(q, x.cuda(), y.cuda(), kg, vg, table.cuda(), lens.cuda(),
                         inv_freq=inv.cuda(), out=out)
        want, kk, vv, _, tolq, tolk = ref.append(q0, x, y, lens.clamp(min=0), None, None, 0, inv,
                                                 False, 1.0, None)
        for n in range(N):
            if lens[n] < 0:
                assert torch.equal(q[n].cpu(), q0[n])
            else:
                assert bool(((q[n].cpu().double() - want[n]).abs() <= tolq[n]).all())
        kc, vc = kg.cpu(), vg.cpu()
        wk, wv, tk = k.double(), v.clone(), torch.zeros(k.shape, dtype=torch.float64)
        for n, r in itertools.product(range(N), range(R)):
            t = int(lens[n]) + r
            if lens[n] < 0 or t // S >= table.shape[1] or table[n, t // S] < 0:
                continue
            p = int(table[n, t // S])
            wk[p, t % S], wv[p, t % S], tk[p, t % S] = kk[n, r], vv[n, r], tolk[n, r]
        assert bool(((kc.double() - wk).abs() <= tk).all()) and torch.equal(vc, wv)
        assert int(out.status.item()) == psi.PSI_DEV_BAD_PAGE


# ---- commit --------------------------------------------------------------------------

def _layers(pool, L, seed):
    return torch.randn((L, *pool.shape), generator=_gen(seed)).to(pool.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,H,D,heads_first", [(16, 2, 64, False), (5, 3, 40, True),
                                               (1, 1, 8, False), (64, 4, 128, True)])
def test_commit_moves_the_accepted_path(S, H, D, heads_first, dtype):
    """Paths of every length, overlapping in place, over page borders."""
    N, M, L = 7, 40, 3
    rng = random.Random(S)
    lens = [0, 1, 17, 130, -1, 63, 64]
    k, v, table, lens = _cache(N, lens, M + 1, H, D, S, dtype, 60, slack=1)
    kl, vl = _layers(k, L, 61), _layers(v, L, 62)
    if heads_first:
        kl, vl = (x.transpose(2, 3).contiguous().transpose(2, 3) for x in (kl, vl))
    n_acc = [0, 1, M, 12, 5, 9, 20]
    path = torch.full((N, M), -1, dtype=torch.int32)
    for n in range(N):
        path[n, :n_acc[n]] = torch.tensor(sorted(rng.sample(range(M), n_acc[n])),
                                          dtype=torch.int32)
    kg, vg = (x.cuda() for x in (kl, vl))
    if heads_first:
        kg, vg = (x.transpose(2, 3).contiguous().cuda().transpose(2, 3) for x in (kl, vl))
    r = psi.cache_commit(kg, vg, table.cuda(), lens.cuda(), path.cuda(),
                         torch.tensor(n_acc, dtype=torch.int32).cuda())
    wk, wv = kl.clone(), vl.clone()
    for n in range(N):
        for j in range(n_acc[n] if lens[n] >= 0 else 0):
            a, b = int(lens[n]) + 1 + int(path[n, j]), int(lens[n]) + 1 + j
            for w, src in ((wk, kl), (wv, vl)):
                w[:, int(table[n, b // S]), b % S] = src[:, int(table[n, a // S]), a % S]
    assert torch.equal(kg.cpu(), wk) and torch.equal(vg.cpu(), wv)
    want = [int(n) if n < 0 else int(n) + 1 + c for n, c in zip(lens, n_acc)]
    assert r.lens.tolist() == want and int(r.status.item()) == 0


def test_commit_bad_paths_and_pages():
    N, M, L, S, H, D = 5, 6, 2, 4, 1, 64
    k, v, table, lens = _cache(N, [3, 3, 3, 3, 3], M + 1, H, D, S, "bf16", 63)
    kl, vl = _layers(k, L, 64), _layers(v, L, 65)
    path = torch.tensor([[1, 3, 3, 5, -1, -1], [4, 2, -1, -1, -1, -1], [0, 1, 2, 3, 4, 5],
                         [1, 6, 7, 8, 9, 10], [2, 4, 5, -1, -1, -1]], dtype=torch.int32)
    n_acc = torch.tensor([4, 2, 9, 3, 3], dtype=torch.int32)
    keep = [2, 1, 6, 1, 3]
    table[4, 2] = -1  # nodes 4 and 5 (positions 8 and 9) have no page: left out
    kg, vg = kl.cuda(), vl.cuda()
    r = psi.cache_commit(kg, vg, table.cuda(), lens.cuda(), path.cuda(), n_acc.cuda())
    wk, wv = kl.clone(), vl.clone()
    for n in range(N):
        for j in range(keep[n]):
            a, b = int(lens[n]) + 1 + int(path[n, j]), int(lens[n]) + 1 + j
            pa, pb = int(table[n, a // S]), int(table[n, b // S])
            if pa >= 0 and pb >= 0:
                wk[:, pb, b % S], wv[:, pb, b % S] = kl[:, pa, a % S], vl[:, pa, a % S]
    assert torch.equal(kg.cpu(), wk) and torch.equal(vg.cpu(), wv)
    assert r.lens.tolist() == [4 + c for c in keep]
    assert int(r.status.item()) == psi.PSI_DEV_BAD_PATH | psi.PSI_DEV_BAD_PAGE


# ---- pages ---------------------------------------------------------------------------------

def _same(state, want):
    assert state.table.tolist() == want.table
    assert state.counts.tolist() == want.counts
    assert state.refs.tolist() == want.refs
    assert int(state.n_free.item()) == want.n_free
    assert state.free.tolist()[:want.n_free] == want.free[:want.n_free]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("N,P,S,mp", [(1, 1, 16, 1), (6, 40, 4, 9), (64, 700, 16, 40),
                                      (1500, 5000, 3, 6)])
def test_resize_and_fork_follow_the_plain_bookkeeping(N, P, S, mp, in_place):
    """Random growth, shrinkage, forks and frees, step by step; some steps ask
    for more than the pool or a row holds."""
    rng = random.Random(N)
    state = psi.PageState.empty(N, mp, P)
    want = ref.Pages(state.table, state.counts, state.refs, state.free, state.n_free)
    lens = [0] * N
    L, H, D = 2, 1, 8
    kp = torch.randn(L, P, S, H, D, generator=_gen(1)).cuda()
    vp = torch.randn(L, P, S, H, D, generator=_gen(2)).cuda()
    for step in range(12):
        before = ref.Pages(state.table, state.counts, state.refs, state.free, state.n_free)
        if step % 3 != 2:
            # a length grows within what is held, or the sequence ends; some are absent
            ask = [rng.choice((0, n, n + 1, min(n + rng.randint(0, 2 * S), mp * S + 2)))
                   for n in lens]
            ask = [-1 if rng.random() < 0.1 else a for a in ask]
            extra = rng.choice((0, 1, S))
            t = torch.tensor(ask, dtype=torch.int32).cuda()
            out = psi.ResizeResult(state, torch.zeros(1, dtype=torch.int32, device="cuda")) \
                if in_place else None
            r = psi.cache_resize(state, t, extra, S, out=out)
            want.resize(ask, extra, S)
            if not in_place:
                _same(state, before)  # the given state is untouched
            state = r.pages
            lens = [n if a < 0 else min(a, c * S) for n, a, c in zip(lens, ask, want.counts)]
            missed = any(a >= 0 and -(-(a + extra) // S) > c for a, c in zip(ask, want.counts))
            assert int(r.status.item()) == (psi.PSI_DEV_NO_PAGES if missed else 0)
        else:
            K = max(1, N // 3)
            src = [rng.randrange(N) for _ in range(K)]
            dst = rng.sample(range(N), K)
            t = torch.tensor(lens, dtype=torch.int32).cuda()
            out = psi.ForkResult(state, t, torch.zeros(1, dtype=torch.int32, device="cuda")) \
                if in_place else None
            k0, v0 = kp.clone(), vp.clone()
            r = psi.cache_fork(kp, vp, state, t, torch.tensor(src, dtype=torch.int32).cuda(),
                               torch.tensor(dst, dtype=torch.int32).cuda(), out=out)
            for a, b, c in want.fork(lens, src, dst, S):
                k0[:, b, :c], v0[:, b, :c] = k0[:, a, :c], v0[:, a, :c]
            assert torch.equal(kp, k0) and torch.equal(vp, v0)
            if not in_place:
                _same(state, before)
            state = r.pages
            assert r.lens.tolist() == lens
        _same(state, want)
    psi.cache_resize(state, torch.zeros(N, dtype=torch.int32, device="cuda"), 0, S,
                     out=psi.ResizeResult(state, r.status))
    assert int(state.n_free.item()) == P and not bool(state.refs.any())
    assert sorted(state.free.tolist()) == list(range(P))


def test_pages_with_errors_in_the_state():
    """Bad table entries, a page released twice, a stack with bad entries, and
    forks that must be left out: flagged, and nothing else is touched."""
    i32 = dict(dtype=torch.int32, device="cuda")
    s = psi.PageState.empty(3, 4, 8)
    s.table[0, :3] = torch.tensor([5, 99, 5], **i32)
    s.counts[0] = 3
    s.refs[5] = 1
    s.free[:] = torch.tensor([0, 1, 2, 3, 4, 6, 7, -1], **i32)
    s.n_free[0] = 7
    r = psi.cache_resize(s, torch.tensor([0, -1, -1], **i32), 0, 16)
    assert int(r.status.item()) == psi.PSI_DEV_BAD_PAGE
    assert r.pages.table[0].tolist() == [-1] * 4 and int(r.pages.n_free.item()) == 8
    assert int(r.pages.free[7].item()) == 5 and not bool(r.pages.refs.any())
    # forks: out of range, onto itself, onto a held row, onto a row twice, a chain
    s = psi.PageState.empty(6, 4, 8)
    lens = torch.tensor([20, 5, 0, 0, 0, -1], **i32)
    s = psi.cache_resize(s, lens, 0, 16).pages
    kp = torch.randn(1, 8, 16, 1, 8, generator=_gen(3)).cuda()
    src = torch.tensor([0, 0, 9, 1, 0, 5], **i32)
    dst = torch.tensor([2, 2, 3, 0, -1, 4], **i32)
    r = psi.cache_fork(kp, kp.clone(), s, lens, src, dst)
    assert int(r.status.item()) == psi.PSI_DEV_BAD_SEQ
    assert r.lens.tolist() == [20, 5, 20, 0, 0, -1]
    assert r.pages.counts.tolist() == [2, 1, 2, 0, 0, 0]
    assert r.pages.table[2, 0] == s.table[0, 0] and r.pages.refs[int(s.table[0, 0])] == 2
    # a length that its pages do not cover
    far = torch.tensor([50, 5, 0, 0, 0, -1], **i32)
    r = psi.cache_fork(kp, kp.clone(), s, far, src[:1], dst[:1])
    assert int(r.status.item()) == psi.PSI_DEV_BAD_PAGE and r.lens[2] == 0


# ---- together ------------------------------------------------------------------------------

class _Model:
    """Two layers of attention over token embeddings, float32 weights."""

    def __init__(self, dt, seed=0, V=97, Hq=4, H=2, D=64, L=2):
        g = _gen(seed)
        w = Hq * D
        self.V, self.Hq, self.H, self.D, self.L = V, Hq, H, D, L
        self.embed = torch.randn(V, w, generator=g)
        self.qkv = [torch.randn(w, (Hq + 2 * H) * D, generator=g) / math.sqrt(w) for _ in range(L)]
        self.out = [torch.randn(w, w, generator=g) / math.sqrt(w) for _ in range(L)]
        self.head = torch.randn(w, V, generator=g) / math.sqrt(w)
        self.qw = (1 + 0.1 * torch.randn(D, generator=g))
        self.inv, self.scale = psi.rope_frequencies(D, 1e4, device="cpu")

    def greedy(self, tokens, steps):
        """Plain decoding in float64: the continuation of `tokens`."""
        tokens = list(tokens)
        for _ in range(steps):
            x = self.embed[tokens].double()
            T = len(tokens)
            pos = torch.arange(T, dtype=torch.float64)
            for l in range(self.L):
                y = (x @ self.qkv[l].double()).view(T, self.Hq + 2 * self.H, self.D)
                q, k, v = y.split((self.Hq, self.H, self.H), dim=1)
                q, k, _, _, _, _ = ref.append(q[:, None].float().double().float(), k[:, None].float(),
                                              v[:, None].float(), pos, self.qw, self.qw, 1e-6,
                                              self.inv, False, 1.0, None)
                q, k = q[:, 0], k[:, 0].repeat_interleave(self.Hq // self.H, 1)
                v = v.repeat_interleave(self.Hq // self.H, 1)
                s = torch.einsum("thd,shd->hts", q, k) / math.sqrt(self.D)
                s = s.masked_fill(torch.ones(T, T).triu(1).bool(), -math.inf)
                o = torch.einsum("hts,shd->thd", s.softmax(-1), v)
                x = x + o.reshape(T, -1) @ self.out[l].double()
            tokens.append(int((x[-1] @ self.head.double()).argmax()))
        return tokens


def test_serving_steps_with_trees_follow_plain_decoding():
    """Tree drafts, append, attend, verify, commit, resize and a fork in the
    middle: the emitted tokens are those of decoding one by one in float64."""
    m = _Model("f32")
    N, live, M, S, mp, P, steps = 3, 2, 12, 4, 30, 80, 22
    R = M + 1
    start = [[3], [50], []]
    truth = [m.greedy(s, steps) if s else [] for s in start]
    rng = random.Random(1)
    kp = torch.zeros(m.L, P, S, m.H, m.D, device="cuda")
    vp = torch.zeros_like(kp)
    pages = psi.PageState.empty(N, mp, P)
    lens = torch.tensor([0, 0, -1], dtype=torch.int32, device="cuda")
    done = [list(s) for s in start]  # tokens so far; the last one is not in the cache yet
    w = {n: getattr(m, n).cuda() for n in ("embed", "head", "qw", "inv")}
    forked = False
    for step in range(12):
        room = psi.cache_resize(pages, lens, R, S)
        assert int(room.status.item()) == 0
        pages = room.pages
        tokens, parents = torch.zeros(N, M, dtype=torch.int32), torch.zeros(N, M, dtype=torch.int32)
        for n in range(N):
            right = truth[n][len(done[n]):] if done[n] else []
            spine = -1  # the last node on the true path
            got = 0
            for k in range(M):
                on = right and got < len(right) and rng.random() < 0.45
                parents[n, k] = spine if on or rng.random() < 0.5 else rng.randint(-1, k - 1)
                tokens[n, k] = right[got] if on else rng.randrange(m.V)
                if on:
                    spine, got = k, got + 1
        par = parents.cuda()
        root = torch.tensor([[d[-1] if d else 0] for d in done], dtype=torch.int32)
        x = w["embed"][torch.cat([root, tokens], 1).long().cuda()]
        for l in range(m.L):
            y = (x @ m.qkv[l].cuda()).view(N, R, m.Hq + 2 * m.H, m.D)
            q, k, v = y.split((m.Hq, m.H, m.H), dim=2)
            a = psi.cache_append(q, k, v, kp[l], vp[l], pages.table, lens, q_weight=w["qw"],
                                 k_weight=w["qw"], inv_freq=w["inv"], parents=par)
            o = psi.attend_block(a.q, kp[l], vp[l], pages.table, lens, parents=par)
            assert int(a.status.item()) == 0 and int(o.status.item()) == 0
            att = o.o.masked_fill((lens < 0)[:, None, None, None], 0)
            x = x + att.reshape(N, R, -1) @ m.out[l].cuda()
        res = psi.verify_tree_greedy((x @ w["head"]).contiguous(), tokens.cuda(), par)
        c = psi.cache_commit(kp, vp, pages.table, lens, res.path_nodes, res.path_len)
        assert int(c.status.item()) == 0
        lens = c.lens
        pages = psi.cache_resize(pages, lens, 0, S).pages
        for n in range(N):
            if int(lens[n]) >= 0:
                emitted = res.tokens[n, :int(res.path_len[n]) + 1].tolist()
                done[n] += emitted
                assert int(lens[n]) == len(done[n]) - 1
        if not forked and len(done[0]) > 5:  # sequence 0 goes on twice
            lens = torch.where(lens < 0, torch.zeros_like(lens), lens)
            f = psi.cache_fork(kp, vp, pages, lens, torch.tensor([0], dtype=torch.int32).cuda(),
                               torch.tensor([2], dtype=torch.int32).cuda())
            assert int(f.status.item()) == 0
            pages, lens, forked = f.pages, f.lens, True
            done[2], truth[2] = list(done[0]), truth[0]
        if min(len(done[n]) for n in range(3 if forked else 2)) >= steps:
            break
    assert forked
    for n in range(N):
        k = min(len(done[n]), len(truth[n]))
        assert k > 8 and done[n][:k] == truth[n][:k], (n, done[n], truth[n])
    freed = psi.cache_resize(pages, torch.zeros_like(lens), 0, S).pages
    assert int(freed.n_free.item()) == P


def test_linear_step_commits_by_its_count():
    """A chain verified by the linear verify: the accepted rows are in place."""
    N, B, S, H, D = 2, 4, 4, 1, 64
    k, v, table, lens = _cache(N, [6, 1], B + 1, H, D, S, "bf16", 90)
    g = _gen(91)
    q = torch.randn(N, B + 1, 2, D, generator=g).bfloat16()
    kg, vg = k.cuda(), v.cuda()
    o1 = psi.attend_block(q.cuda(), kg, vg, table.cuda(), lens.cuda()).o
    logits = torch.randn(N, B + 1, 64, generator=g).cuda()
    ids = logits[:, :B].argmax(-1).int()
    ids[0, 2] = (ids[0, 2] + 1) % 64
    n = psi.verify_linear(logits, None, ids.contiguous(), 0.0).n_emitted
    assert n.tolist() == [3, 5]
    # row 2 of sequence 0 read again as a step of one token after two kept rows
    lens2 = (lens.cuda() + n - 1).contiguous()
    one = torch.stack([q[0, 2:3], q[1, 4:5]]).cuda()
    o2 = psi.attend_block(one, kg, vg, table.cuda(), lens2).o
    # both round the same sum: half a step of the output and of the weights each, 4 * 2^-8 of
    # sum p |v|, which stays below max |v| < 5
    for n, r in ((0, 2), (1, 4)):
        assert float((o2[n, 0].float() - o1[n, r].float()).abs().max()) <= 5 * 4 * 2.0 ** -8
