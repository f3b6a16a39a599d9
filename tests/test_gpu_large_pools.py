"""Page bookkeeping with more pages than fit one CTA's shared memory (49,152),
where the reference counts are worked on in place."""
import random

import pytest
import torch

import cache_reference as ref
import rejection_sampling_verify_b200 as psi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("N,P,S,mp", [(5, 49152, 16, 20000), (5, 49153, 16, 20000),
                                      (40, 60001, 4, 3000), (1100, 50000, 2, 60)])
def test_large_pools_follow_the_plain_bookkeeping(N, P, S, mp, in_place):
    rng = random.Random(P + N)
    s = psi.PageState.empty(N, mp, P)
    want = ref.Pages(s.table, s.counts, s.refs, s.free, s.n_free)
    lens = [0] * N
    pool = torch.zeros(1, P, S, 1, 8, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(5):
        if step == 2:
            K = max(1, N // 4)
            src, dst = [rng.randrange(N) for _ in range(K)], rng.sample(range(N), K)
            t = torch.tensor(lens, dtype=torch.int32).cuda()
            r = psi.cache_fork(pool, pool.clone(), s, t, torch.tensor(src, dtype=torch.int32).cuda(),
                               torch.tensor(dst, dtype=torch.int32).cuda(),
                               out=psi.ForkResult(s, t, word) if in_place else None)
            want.fork(lens, src, dst, S)
            assert r.lens.tolist() == lens
        else:
            ask = [rng.choice((0, n, rng.randint(0, mp * S))) if step < 4 else 0 for n in lens]
            t = torch.tensor(ask, dtype=torch.int32).cuda()
            r = psi.cache_resize(s, t, 0, S, out=psi.ResizeResult(s, word) if in_place else None)
            want.resize(ask, 0, S)
            lens = [min(a, c * S) for a, c in zip(ask, want.counts)]
        s = r.pages
        assert s.table.tolist() == want.table and s.counts.tolist() == want.counts
        assert s.refs.tolist() == want.refs and int(s.n_free.item()) == want.n_free
        assert s.free.tolist()[:want.n_free] == want.free[:want.n_free]
    assert int(s.n_free.item()) == P and not bool(s.refs.any())
