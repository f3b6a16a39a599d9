"""A whole serving step of the cache's calls captured into a graph, replayed on
new inputs between ordinary calls; and steps on two streams at once."""
import pytest
import torch

import rejection_sampling_verify_b200 as psi

pytestmark = pytest.mark.gpu

N, M, Hq, H, D, S, L, P, MP, V = 4, 6, 8, 2, 64, 16, 2, 64, 12, 50
R = M + 1
I32 = dict(dtype=torch.int32, device="cuda")


class Step:
    """Buffers of one stream of steps, and the step over them."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.k, self.v = (torch.zeros(L, P, S, H, D, dtype=torch.bfloat16, device="cuda")
                          for _ in range(2))
        self.qkv = torch.zeros(L, N, R, Hq + 2 * H, D, dtype=torch.bfloat16, device="cuda")
        self.logits = torch.zeros(N, R, V, device="cuda")
        self.tokens = torch.zeros(N, M, **I32)
        self.parents = torch.full((N, M), -1, **I32)
        self.lens = torch.zeros(N, **I32)
        self.inv, _ = psi.rope_frequencies(D)
        self.pages = psi.PageState.empty(N, MP, P)
        self.src, self.dst = torch.tensor([0], **I32), torch.tensor([N - 1], **I32)

    def renew(self, lens):
        """New inputs in the same buffers."""
        for t in (self.k, self.v, self.qkv):
            t.copy_(torch.randn(t.shape, generator=self.g, device="cuda"))
        self.logits.copy_(torch.randn(self.logits.shape, generator=self.g, device="cuda"))
        up = torch.rand(N, M, generator=self.g, device="cuda") * torch.arange(1, M + 1, device="cuda")
        self.parents.copy_(up.int() - 1)
        rows = self.logits.argmax(-1)  # about half of the nodes continue their parents
        follow = torch.rand(N, M, generator=self.g, device="cuda") < 0.5
        self.tokens.copy_(torch.where(follow, rows.gather(1, self.parents.long() + 1), 0))
        self.lens.copy_(torch.tensor(lens))
        # row N - 1 is empty; the others' pages go as their lengths do
        fresh = psi.PageState.empty(N, MP, P)
        room = psi.cache_resize(fresh, self.lens.clamp(min=0), 0, S).pages
        for name in ("table", "counts", "refs", "free", "n_free"):
            getattr(self.pages, name).copy_(getattr(room, name))

    def run(self):
        room = psi.cache_resize(self.pages, self.lens, R, S)
        outs, words = [], [room.status]
        for l in range(L):
            q, k, v = self.qkv[l].split((Hq, H, H), dim=2)
            a = psi.cache_append(q, k, v, self.k[l], self.v[l], room.pages.table, self.lens,
                                 inv_freq=self.inv, parents=self.parents)
            o = psi.attend_block(a.q, self.k[l], self.v[l], room.pages.table, self.lens,
                                 parents=self.parents, want_lse=True)
            outs += [a.q[:-1], o.o[:-1], o.lse[:-1]]  # (the last sequence is absent)
            words += [a.status, o.status]
        t = psi.verify_tree_greedy(self.logits, self.tokens, self.parents)
        c = psi.cache_commit(self.k, self.v, room.pages.table, self.lens, t.path_nodes, t.path_len)
        z = psi.cache_resize(room.pages, c.lens, 0, S)
        f = psi.cache_fork(self.k, self.v, z.pages, c.lens, self.src, self.dst)
        words += [c.status, z.status, f.status]
        p = f.pages
        return outs + [t.tokens, f.lens, p.table, p.counts, p.refs, p.n_free, self.k, self.v] + words


def _copy(ts):
    return [t.clone() for t in ts]


LENS = ([20, 3, 100, -1], [0, 1, 15, -1], [16, 128, 31, -1])


def test_a_captured_step_follows_the_plain_one():
    s = Step(1)
    s.renew(LENS[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = s.run()
    for lens in LENS:
        s.renew(lens)
        k, v = s.k.clone(), s.v.clone()
        want = _copy(s.run())
        for _ in range(2):
            s.k.copy_(k)
            s.v.copy_(v)
            g.replay()
            for a, b in zip(got, want):
                assert torch.equal(a, b)
        assert all(int(w) == 0 for w in want[-8:])
        assert int(want[-len(want) + 3 * L + 1][N - 1]) > 0  # the fork was made


def test_steps_on_two_streams_at_once():
    one, two = Step(2), Step(3)
    for lens in LENS:
        want, start = [], []
        for s in (one, two):
            s.renew(lens)
            start.append((s.k.clone(), s.v.clone()))
            want.append(_copy(s.run()))
            s.k.copy_(start[-1][0])
            s.v.copy_(start[-1][1])
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        got = [None, None]
        for _ in range(3):
            for i, s in enumerate((one, two)):
                with torch.cuda.stream(streams[i]):
                    s.k.copy_(start[i][0])
                    s.v.copy_(start[i][1])
                    got[i] = s.run()
        torch.cuda.synchronize()
        for a, b in zip(got[0] + got[1], want[0] + want[1]):
            assert torch.equal(a, b)
