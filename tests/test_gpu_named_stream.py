"""Calls on a named stream while the current one takes and writes memory."""
import pytest
import torch

import rejection_sampling_verify_b200 as psi

pytestmark = pytest.mark.gpu


def _fill():
    """Takes blocks of every usual size on the current stream and writes them."""
    for size in (512, 1 << 12, 1 << 16, 1 << 18, 1 << 20, 1 << 22):
        for _ in range(6):
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")


def _behind(s, call):
    """The call's result on `s`, which is kept busy for some 20 ms meanwhile."""
    call(s)  # (the allocator has blocks of these sizes to hand out)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(40_000_000)
    r = call(s)
    _fill()
    torch.cuda.synchronize()
    return r


def test_attend_on_a_busy_stream():
    N, R, Hq, H, D, S, n = 1, 5, 8, 2, 128, 16, 5000
    g = torch.Generator().manual_seed(1)
    held = -(-(n + R) // S)
    k, v = (torch.randn(held, S, H, D, generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn(N, R, Hq, D, generator=g).bfloat16().cuda()
    table = torch.arange(held, dtype=torch.int32, device="cuda").view(1, held)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    want = psi.attend_block(q, k, v, table, lens, want_lse=True)
    s = torch.cuda.Stream()
    got = _behind(s, lambda s: psi.attend_block(q, k, v, table, lens, want_lse=True, stream=s))
    assert torch.equal(got.o, want.o) and torch.equal(got.lse, want.lse)
    assert int(got.status.item()) == 0
    out = psi.AttendResult(torch.empty_like(q), None, torch.zeros_like(lens))
    _behind(s, lambda s: psi.attend_block(q, k, v, table, lens, stream=s, out=out))
    assert torch.equal(out.o, want.o)


def test_pages_on_a_busy_stream():
    N, S, L, P = 64, 16, 2, 400
    g = torch.Generator().manual_seed(2)
    pool = torch.randn(L, P, S, 1, 64, generator=g).bfloat16().cuda()
    lens = torch.zeros(2 * N, dtype=torch.int32)
    lens[:N] = torch.randint(1, 60, (N,), generator=g, dtype=torch.int32)
    lens = lens.cuda()
    src = torch.arange(N, dtype=torch.int32, device="cuda")
    dst = src + N

    def step(stream, busy):
        k, v = pool.clone(), pool.clone()
        room = psi.cache_resize(psi.PageState.empty(2 * N, 4, P), lens, 0, S)
        torch.cuda.synchronize()
        if busy:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(40_000_000)
        r = psi.cache_fork(k, v, room.pages, lens, src, dst, stream=stream)
        again = psi.cache_resize(r.pages, r.lens, 1, S, stream=stream)
        if busy:
            _fill()
        torch.cuda.synchronize()
        return k, v, r, again

    want = step(None, False)
    s = torch.cuda.Stream()
    step(s, False)  # (the allocator has blocks of these sizes to hand out)
    k, v, r, again = step(s, True)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    for a, b in ((r, want[2]), (again, want[3])):
        for f in ("table", "counts", "refs", "n_free"):
            assert torch.equal(getattr(a.pages, f), getattr(b.pages, f)), f
        assert int(a.status.item()) == 0
    assert torch.equal(r.lens, want[2].lens)


def test_verify_on_a_busy_stream():
    N, B, V = 3, 4, 1000
    g = torch.Generator().manual_seed(3)
    ar = torch.randn(N, B + 1, V, generator=g).cuda()
    draft = torch.randn(N, B, V, generator=g).cuda()
    ids = torch.randint(0, V, (N, B), generator=g, dtype=torch.int32).cuda()
    parents = torch.tensor([[-1, 0, -1, 2]] * N, dtype=torch.int32).cuda()
    calls = [lambda s: psi.verify_linear(ar, draft, ids, 0.8, 0.9, seed=5, stream=s),
             lambda s: psi.verify_linear(ar, draft, ids, 0.8, seed=5, top_k=20, stream=s),
             lambda s: psi.verify_linear(ar, None, ids, 0.0, stream=s),
             lambda s: psi.verify_tree_greedy(ar, ids, parents, stream=s),
             lambda s: psi.verify_tree_sampled(ar, ids, parents, 0.8, seed=6, stream=s)]
    s = torch.cuda.Stream()
    for call in calls:
        want, got = call(None), _behind(s, call)
        for name, t in vars(want).items():
            if t is not None:
                assert torch.equal(getattr(got, name), t), name
    u = psi.rng_uniforms(7, N, 1, B, psi.PSI_PURPOSE_ACCEPT)
    got = _behind(s, lambda s: psi.rng_uniforms(7, N, 1, B, psi.PSI_PURPOSE_ACCEPT, stream=s))
    assert torch.equal(got, u)
