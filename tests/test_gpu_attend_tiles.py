"""Block attention at every size of its tiles: 16 to 80 packed rows in one
group, 96 to 160 in two, heads that fill a tile's 64 or 128 elements and heads
that end inside a warp, pages that are loaded as boxes and row by row."""
import math

import pytest
import torch

import rejection_sampling_verify_b200 as psi

pytestmark = pytest.mark.gpu

# rows of the block, query heads per kv head
ROWS = [(16, 1), (4, 8), (45, 1), (7, 7), (16, 4), (13, 5), (10, 8), (27, 3), (12, 8), (32, 4),
        (20, 8), (23, 7), (48, 4)]
LENS = [0, 1, 127, 300, 511, 400]
S2N = 2.0 ** -24


def _exact(q, k, v, seen, scale):
    """(o, lse, tol) of one sequence in float64.  The bound: half a step of the
    output and of each weight (2^-8), D + 2 roundings of the score's terms in
    its exponent (twice, for numerator and denominator), 16 for the powers of
    two and products, one for each position of the sum."""
    R, Hq, D = q.shape
    T, H, _ = k.shape
    q, k, v = q.double().view(R, H, Hq // H, D), k.double(), v.double()
    s = torch.einsum("rhgd,thd->rhgt", q, k) * scale
    s = s.masked_fill(~seen[:, None, None, :], -math.inf)
    p = s.softmax(-1)
    o = torch.einsum("rhgt,thd->rhgd", p, v)
    size = torch.einsum("rhgd,thd->rhgt", q.abs(), k.abs()).amax(-1) * scale
    err = 4 * (D + 2) * S2N * size + (T + 16) * S2N + 2.0 ** -8
    tol = 2.0 ** -8 * o.abs() + err[..., None] * torch.einsum("rhgt,thd->rhgd", p, v.abs()) + 1e-30
    return o.reshape(R, Hq, D), s.logsumexp(-1).reshape(R, Hq), tol.reshape(R, Hq, D)


@pytest.mark.parametrize("S", [16, 5])
@pytest.mark.parametrize("D", [64, 128, 40, 72])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("R,G", ROWS)
def test_every_tile_size(R, G, tree, D, S):
    """Enough heads that a CTA works through several tiles (its stages are
    used again); what no sequence holds is NaN."""
    H, N, dev = 32, len(LENS), "cuda"
    g = torch.Generator(device=dev).manual_seed(1000 * R + 10 * D + S)
    held = [-(-(n + R) // S) for n in LENS]
    P = sum(held) + 1
    k, v = (torch.randn(P, S, H, D, generator=g, device=dev).bfloat16() for _ in range(2))
    q = torch.randn(N, R, H * G, D, generator=g, device=dev).bfloat16()
    order = torch.randperm(P, generator=g, device=dev).to(torch.int32)
    table = torch.full((N, max(held)), -1, dtype=torch.int32, device=dev)
    at, free = 0, torch.ones(P, S, dtype=torch.bool, device=dev)
    where = []
    for n, count in enumerate(held):
        table[n, :count] = order[at:at + count]
        at += count
        t = torch.arange(LENS[n] + R, device=dev)
        where.append((table[n].long()[t // S], t % S))
        free[where[n]] = False
    k[free] = math.nan
    v[free] = math.nan
    lens = torch.tensor(LENS, dtype=torch.int32, device=dev)
    parents = None
    sees = torch.ones(R, R, dtype=torch.bool).tril().repeat(N, 1, 1)
    if tree and R > 1:
        cpu = torch.Generator().manual_seed(R)
        up = [[int(torch.randint(max(-1, i - 9), i, (1,), generator=cpu)) for i in range(R - 1)]
              for _ in range(N)]
        parents = torch.tensor(up, dtype=torch.int32, device=dev)
        sees = torch.eye(R, dtype=torch.bool).repeat(N, 1, 1)
        for n in range(N):
            for r in range(1, R):
                sees[n, r] |= sees[n, up[n][r - 1] + 1]
    got = psi.attend_block(q, k, v, table, lens, parents=parents, want_lse=True)
    assert int(got.status.item()) == 0
    for n in range(N):
        seen = torch.cat([torch.ones(R, LENS[n], dtype=torch.bool), sees[n]], 1).to(dev)
        o, lse, tol = _exact(q[n], k[where[n]], v[where[n]], seen, D ** -0.5)
        err = (got.o[n].double() - o).abs()
        assert bool((err <= tol).all()), (n, float((err / tol).max()))
        # the score's rounding (below 2^-12 at these sizes) and the sum's
        assert bool(((got.lse[n].double() - lse).abs() <= 2.0 ** -12 + 1e-6 * lse.abs()).all())
