"""Page states whose stack of free pages is wrong: a popped entry that is not
a free page is left out, and nobody else's page changes hands."""
import pytest
import torch

import rejection_sampling_verify_b200 as psi

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def _state(N, max_pages, P, held, stack):
    """A state with held[n] = pages of row n, and `stack` as it is (its top last)."""
    s = psi.PageState.empty(N, max_pages, P)
    for n, row in enumerate(held):
        for i, p in enumerate(row):
            s.table[n, i] = p
            s.refs[p] += 1
        s.counts[n] = len(row)
    s.free[:len(stack)] = torch.tensor(stack, **I32)
    s.n_free[0] = len(stack)
    return s


# up to 49,152 pages the counts are worked on in shared memory, above in place
@pytest.mark.parametrize("P", [8, 60000])
def test_resize_leaves_out_what_is_no_free_page(P):
    """Popped in turn: -1, past the pool, a page that two rows hold, a free
    page, and the same one again."""
    for _ in range(5):  # (the first of two takers gets a page, every time)
        s = _state(7, 3, P, [[3], [3], [5]], [6, 6, 3, P, -1])
        lens = torch.tensor([16, 16, 16, 32, 16, 16, 16], **I32)
        r = psi.cache_resize(s, lens, 0, 16)
        assert int(r.status.item()) == psi.PSI_DEV_BAD_PAGE
        assert r.pages.table.tolist() == [[3, -1, -1], [3, -1, -1], [5, -1, -1], [-1, -1, -1],
                                          [-1, -1, -1], [6, -1, -1], [-1, -1, -1]]
        assert r.pages.counts.tolist() == [1, 1, 1, 2, 1, 1, 1]
        refs = r.pages.refs.tolist()
        assert (refs[3], refs[5], refs[6], sum(refs)) == (2, 1, 1, 4)
        assert int(r.pages.n_free.item()) == 0
    # and the page that two rows hold is given back only by the second of them
    a = psi.cache_resize(r.pages, torch.tensor([0, -1, -1, -1, -1, -1, -1], **I32), 0, 16)
    assert int(a.status.item()) == 0 and int(a.pages.n_free.item()) == 0
    b = psi.cache_resize(a.pages, torch.tensor([0, 0, -1, -1, -1, -1, -1], **I32), 0, 16)
    assert int(b.status.item()) == 0 and b.pages.free[:1].tolist() == [3]


def test_one_row_that_pops_a_page_again_and_again_gets_it_once():
    s = _state(1, 40, 40, [], [4] * 33)
    r = psi.cache_resize(s, torch.tensor([33 * 4], **I32), 0, 4)
    assert int(r.status.item()) == psi.PSI_DEV_BAD_PAGE
    assert r.pages.table[0].tolist() == [4] + [-1] * 39
    assert r.pages.refs.tolist() == [int(p == 4) for p in range(40)]


@pytest.mark.parametrize("P", [8, 60000])
def test_fork_leaves_out_what_is_no_free_page(P):
    """Popped in turn: a page that two rows hold, a free page, the same one
    again, and -1: one fork is made."""
    kp = torch.randn(1, P, 4, 1, 8, generator=torch.Generator().manual_seed(1)).cuda()
    before = kp.clone()
    for _ in range(5):
        s = _state(7, 2, P, [[3, 5], [3]], [-1, 6, 6, 3])
        lens = torch.tensor([6, 4, 0, 0, 0, 0, 0], **I32)
        r = psi.cache_fork(kp, kp.clone(), s, lens, torch.tensor([0, 0, 0, 0], **I32),
                           torch.tensor([2, 3, 4, 5], **I32))
        assert int(r.status.item()) == psi.PSI_DEV_BAD_PAGE
        assert r.lens.tolist() == [6, 4, 0, 6, 0, 0, 0]
        assert r.pages.counts.tolist() == [2, 1, 0, 2, 0, 0, 0]
        assert r.pages.table[3].tolist() == [3, 6]
        refs = r.pages.refs.tolist()
        assert (refs[3], refs[5], refs[6], sum(refs)) == (3, 1, 1, 5)
        assert int(r.pages.n_free.item()) == 0
    before[0, 6, :2] = before[0, 5, :2]  # the partial page's two slots
    assert torch.equal(kp, before)
