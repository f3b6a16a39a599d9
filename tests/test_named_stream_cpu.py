"""A call that names a stream takes all its memory on that stream.

Memory from the current stream would go back to the allocator when the call
returns, and to the next allocation there, while the call's kernels on the
named stream have still to use it.  Seen here without a GPU: the calls run on
host tensors with the launches recorded, and every allocation has to happen
inside the named stream's context."""
import contextlib

import pytest
import torch

import rejection_sampling_verify_b200 as psi
from rejection_sampling_verify_b200 import cache


class Named:
    """Stands in for a torch.cuda.Stream."""
    cuda_stream = 0x77


@pytest.fixture
def made(monkeypatch):
    """Allocations made by the call under test: (bytes, stream they were made on)."""
    log, on = [], [None]

    @contextlib.contextmanager
    def stream(s):
        before, on[0] = on[0], s if s is not None else on[0]
        yield
        on[0] = before

    def raw(dev=None):
        return 0 if on[0] is None else on[0].cuda_stream

    def recorded(f):
        def g(*a, **k):
            k.pop("device", None)
            t = f(*a, **k)
            log.append((t.numel() * t.element_size(), on[0]))
            return t
        return g

    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda *a: Named() if on[0] is not None else type("D", (), {"cuda_stream": 0}))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device=None: Named())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", raw, raising=False)
    monkeypatch.setattr(cache, "_on_device", lambda ref, named: 0)
    monkeypatch.setattr(psi, "_device_of", lambda ref, **t: torch.device("cpu"))
    # (the compiled binding does not take host tensors)
    monkeypatch.setattr(cache, "_short", lambda: type("S", (), dict.fromkeys(
        ("append", "attend", "commit", "resize", "fork"), staticmethod(lambda *a: None))))
    monkeypatch.setattr(cache, "_binding", None)
    launched = []
    for mod, names in ((cache, ("psi_cache_append", "psi_attend_block", "psi_cache_commit",
                                "psi_cache_resize", "psi_cache_fork")),
                       (psi, ("psi_verify_linear", "psi_verify_linear_topk",
                              "psi_verify_tree_greedy", "psi_verify_tree_sampled",
                              "psi_rng_uniforms"))):
        for name in names:
            monkeypatch.setattr(mod, name, lambda *a, name=name: launched.append((name, a[-1])) or 0)
    return log, launched


N, R, Hq, H, D, S, P, L, M, V = 2, 3, 4, 2, 64, 16, 8, 2, 4, 32


def _inputs():
    i32 = torch.int32
    return dict(
        q=torch.ones(N, R, Hq, D).bfloat16(), k=torch.ones(N, R, H, D).bfloat16(),
        pool=torch.ones(L, P, S, H, D).bfloat16(), table=torch.ones(N, 4).to(i32),
        lens=torch.ones(N).to(i32), path=torch.ones(N, M).to(i32), src=torch.ones(1).to(i32),
        pages=psi.PageState(torch.ones(N, 4).to(i32), torch.ones(N).to(i32), torch.ones(P).to(i32),
                            torch.ones(P).to(i32), torch.ones(1).to(i32)),
        logits=torch.ones(N, M + 1, V), draft=torch.ones(N, M, V))


CALLS = {
    "append": lambda t, s: psi.cache_append(t["q"], t["k"], t["k"], t["pool"][0], t["pool"][0],
                                            t["table"], t["lens"], stream=s),
    "attend": lambda t, s: psi.attend_block(t["q"], t["pool"][0], t["pool"][0], t["table"],
                                            t["lens"], want_lse=True, stream=s),
    "attend_out": lambda t, s: psi.attend_block(
        t["q"], t["pool"][0], t["pool"][0], t["table"], t["lens"], stream=s,
        out=psi.AttendResult(t["q"].clone(), None, t["src"].clone())),
    "commit": lambda t, s: psi.cache_commit(t["pool"], t["pool"], t["table"], t["lens"], t["path"],
                                            t["lens"], stream=s),
    "resize": lambda t, s: psi.cache_resize(t["pages"], t["lens"], 0, S, stream=s),
    "fork": lambda t, s: psi.cache_fork(t["pool"], t["pool"], t["pages"], t["lens"], t["src"],
                                        t["src"], stream=s),
    "fork_out": lambda t, s: psi.cache_fork(
        t["pool"], t["pool"], t["pages"], t["lens"], t["src"], t["src"], stream=s,
        out=psi.ForkResult(t["pages"], t["lens"], t["src"].clone())),
    "linear": lambda t, s: psi.verify_linear(t["logits"], t["draft"], t["path"], 0.7, stream=s),
    "linear_topk": lambda t, s: psi.verify_linear(t["logits"], t["draft"], t["path"], 0.7,
                                                  want_probs=False, top_k=3, stream=s),
    "linear_out": lambda t, s: psi.verify_linear(
        t["logits"], None, t["path"], 0.0, stream=s,
        out=psi.LinearResult(t["path"].new_ones(N, M + 1), t["lens"].clone(), None, None,
                             t["src"].clone())),
    "tree_greedy": lambda t, s: psi.verify_tree_greedy(t["logits"], t["path"], t["path"], stream=s),
    "tree_sampled": lambda t, s: psi.verify_tree_sampled(t["logits"], t["path"], t["path"], 0.7,
                                                         stream=s),
    "uniforms": lambda t, s: psi.rng_uniforms(1, N, 2, 3, psi.PSI_PURPOSE_ACCEPT, stream=s),
}


@pytest.mark.parametrize("call", CALLS)
def test_memory_of_a_call_on_a_named_stream(call, made):
    log, launched = made
    t, s = _inputs(), Named()
    CALLS[call](t, s)
    assert launched and all(raw == s.cuda_stream for _, raw in launched)
    assert log and all(on is s for _, on in log), log
    log.clear()
    CALLS[call](t, None)  # and on the current one without a name
    assert log and all(on is None for _, on in log), log
