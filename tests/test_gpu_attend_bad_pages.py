"""Sequences of several tiles with pages missing among them, in every shape of
a CTA's stages: what lies where a page is missing has no influence, and a tile
before it keeps its values."""
import pytest
import torch

import rejection_sampling_verify_b200 as psi

pytestmark = pytest.mark.gpu

S2N = 2.0 ** -24


# packed rows of 16, 32, 48, 64 and 80 in one group; 48, 64 and 80 in two
@pytest.mark.parametrize("R,G", [(1, 8), (8, 2), (17, 1), (9, 4), (3, 16), (16, 4), (10, 8),
                                 (12, 8), (32, 4), (20, 8)])
@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("S", [16, 32, 5])
def test_missing_pages_among_many_tiles(R, G, D, S):
    """Every run gives the same bits, and those of the definition (the bound is
    that of tests/cache_reference.py)."""
    N, H, dev = 20, 2, "cuda"
    g = torch.Generator(device=dev).manual_seed(100 * R + D + S)
    lens = torch.randint(500, 3000, (N,), generator=g, device=dev).tolist()
    held = [-(-(n + R) // S) for n in lens]
    P = sum(held)
    k, v = (torch.randn(P, S, H, D, generator=g, device=dev).bfloat16() for _ in range(2))
    q = torch.randn(N, R, H * G, D, generator=g, device=dev).bfloat16()
    order = torch.randperm(P, generator=g, device=dev).to(torch.int32)
    table = torch.full((N, max(held)), -1, dtype=torch.int32, device=dev)
    at = 0
    for n, count in enumerate(held):
        table[n, :count] = order[at:at + count]
        at += count
        if n % 4:  # some pages are missing, of most sequences
            gone = torch.randint(0, count, (n % 4 * 2,), generator=g, device=dev)
            table[n, gone] = -1 if n % 2 else P
    t = torch.tensor(lens, dtype=torch.int32, device=dev)
    first = psi.attend_block(q, k, v, table, t)
    assert int(first.status.item()) == psi.PSI_DEV_BAD_PAGE
    for _ in range(25):
        again = psi.attend_block(q, k, v, table, t)
        assert torch.equal(first.o, again.o)
    for n in range(N):
        x = torch.arange(lens[n] + R, device=dev)
        page = table[n].long()[x // S]
        seen = (x[None] <= lens[n] + torch.arange(R, device=dev)[:, None]) & \
            ((page >= 0) & (page < P))[None]
        kk, vv = (p[page.clamp(0, P - 1), x % S].double() for p in (k, v))
        qq = q[n].double().view(R, H, G, D)
        s = torch.einsum("rhgd,thd->rhgt", qq, kk) * D ** -0.5
        p = s.masked_fill(~seen[:, None, None], -torch.inf).softmax(-1)
        o = torch.einsum("rhgt,thd->rhgd", p, vv)
        size = torch.einsum("rhgd,thd->rhgt", qq.abs(), kk.abs()).amax(-1) * D ** -0.5
        err = 4 * (D + 2) * S2N * size + (len(x) + 16) * S2N + 2.0 ** -8
        tol = 2.0 ** -8 * o.abs() + err[..., None] * torch.einsum("rhgt,thd->rhgd", p, vv.abs())
        assert bool(((first.o[n].double().view(R, H, G, D) - o).abs() <= tol).all()), n
