"""The status words of the cache's calls: each is its call's own, made for
ordinary use, on the stream of the call."""
import pytest
import torch

import rejection_sampling_verify_b200 as psi

pytestmark = pytest.mark.gpu


def _resize(**kw):
    pages = psi.PageState.empty(2, 4, 8)
    return psi.cache_resize(pages, torch.tensor([20, 3], dtype=torch.int32, device="cuda"), 1, 16,
                            **kw)


def test_status_words_after_a_call_in_inference_mode():
    """A result of any later call can be used again as `out`."""
    with torch.cuda.stream(torch.cuda.Stream()):
        with torch.inference_mode():
            assert int(_resize().status.item()) == 0
        for _ in range(300):  # more calls than words are zeroed at a time
            r = _resize()
            r.status.zero_()
            assert not r.status.is_inference()


def test_status_words_of_streams_that_are_not_torchs():
    """A stream made elsewhere may be destroyed and its handle used again, so
    nothing is kept for it."""
    own = torch.cuda.Stream()
    seen = set()
    for _ in range(3):
        with torch.cuda.stream(torch.cuda.ExternalStream(own.cuda_stream)):
            r = _resize()
        assert r.status.untyped_storage().nbytes() == 4
        own.synchronize()
        assert int(r.status.item()) == 0
        seen.add(r.status.data_ptr())
    assert seen


def test_status_words_are_not_shared():
    words = [_resize().status for _ in range(600)]
    assert len({w.data_ptr() for w in words}) == 600
    assert not any(int(w) for w in torch.cat(words).tolist())


def test_status_words_of_captured_calls_are_zeroed_on_every_replay():
    pages = psi.PageState.empty(2, 4, 8)
    lens = torch.tensor([20, 3], dtype=torch.int32, device="cuda")
    psi.cache_resize(pages, lens, 1, 16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = psi.cache_resize(pages, lens, 1, 16)
    lens[0] = 1000  # more than a row holds
    g.replay()
    assert int(r.status.item()) == psi.PSI_DEV_NO_PAGES
    lens[0] = 20
    g.replay()
    assert int(r.status.item()) == 0
