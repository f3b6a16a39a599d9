"""Heads that hold infinities, NaN or negative zeros through cache_append:
an element that is not turned is stored as it is, whatever lies beside it."""
import itertools
import math

import pytest
import torch

import rejection_sampling_verify_b200 as psi

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
Hq, H = 4, 2


def _same(a, b):
    """Equal bit for bit, any NaN being like any other."""
    return bool(((a == b) & (a.signbit() == b.signbit()) | (a.isnan() & b.isnan())).all())


def _run(q, k, v, rot, interleaved, weight=None, lens=7):
    N, R, D = q.shape[0], q.shape[1], q.shape[3]
    S = 16
    held = -(-(lens + R) // S)
    kp, vp = (torch.zeros(N * held, S, H, D, dtype=q.dtype, device="cuda") for _ in range(2))
    table = torch.arange(N * held, dtype=torch.int32, device="cuda").view(N, held)
    n = torch.full((N,), lens, dtype=torch.int32, device="cuda")
    inv = psi.rope_frequencies(rot)[0] if rot else None
    r = psi.cache_append(q, k, v, kp, vp, table, n, q_weight=weight, k_weight=weight,
                         inv_freq=inv, interleaved=interleaved)
    assert int(r.status.item()) == 0
    flat = lambda p: p.view(N, held * S, H, D)[:, lens:lens + R]  # noqa: E731
    return r.q, flat(kp), flat(vp)


# (D, rotary_dim): heads of whole chunks, and (40) those taken element by element
SIZES = [(64, 0), (64, 32), (128, 0), (128, 64), (128, 16), (96, 48), (256, 128), (40, 0), (40, 18)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N", [2, 450])  # one and two rows a CTA
@pytest.mark.parametrize("D,rot", SIZES)
def test_what_is_not_turned_is_stored_as_it_is(D, rot, N, interleaved, dtype):
    R = 3
    g = torch.Generator().manual_seed(D + rot)
    q, k, v = (torch.randn(N, R, h, D, generator=g).to(DT[dtype]).cuda() for h in (Hq, H, H))
    clean = _run(q, k, v, rot, interleaved)
    for x in (q, k, v):
        for at, value in ((rot, math.inf), (rot + 5, math.nan), (rot + 9, -math.inf),
                          (D - 1, -0.0), (rot + 8, -0.0)):
            x[0, 1, 1, at] = value
        x[1, 2, :, D - 2] = math.nan
    got = _run(q, k, v, rot, interleaved)
    for x, y, c in zip((q, k, v), got, clean):
        assert _same(y[..., rot:], x[..., rot:])
        assert torch.equal(y[..., :rot], c[..., :rot])  # the turned ones do not see it
    assert _same(got[2], v)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 64), (128, 128), (64, 32), (40, 18)])
def test_a_pair_that_is_turned_keeps_its_infinity_to_itself(D, rot, interleaved, dtype):
    N, R = 2, 2
    g = torch.Generator().manual_seed(D)
    q, k, v = (torch.randn(N, R, h, D, generator=g).to(DT[dtype]).cuda() for h in (Hq, H, H))
    clean = _run(q, k, v, rot, interleaved)
    i = 3  # the pair
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    q[..., a], k[..., b] = math.inf, math.nan
    got = _run(q, k, v, rot, interleaved)
    rest = [d for d in range(D) if d not in (a, b)]
    for y, c in zip(got[:2], clean[:2]):
        assert torch.equal(y[..., rest], c[..., rest])
        assert not bool(y[..., [a, b]].isfinite().any())


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,rot,interleaved", list(itertools.product((64, 128), (0, 32),
                                                                      (False, True))))
def test_the_norm_of_a_head_with_an_infinity(D, rot, interleaved, dtype):
    """x / sqrt(mean x^2 + eps) is 0 for the finite elements and NaN for the
    infinite one, wherever it lies; other heads go on as they were."""
    q, k, v = (torch.randn(2, 2, h, D, generator=torch.Generator().manual_seed(h))
               .to(DT[dtype]).cuda() for h in (Hq, H, H))
    w = torch.full((D,), 1.5, dtype=DT[dtype], device="cuda")
    clean = _run(q, k, v, rot, interleaved, w)
    q[1, 0, 2, D - 3] = k[0, 1, 1, D - 3] = math.inf
    got = _run(q, k, v, rot, interleaved, w)
    for y, c, (n, r, h) in zip(got[:2], clean[:2], ((1, 0, 2), (0, 1, 1))):
        head = y[n, r, h].clone()
        assert bool(head[D - 3].isnan())
        head[D - 3] = 0
        assert not bool(head.any())
        y[n, r, h] = c[n, r, h]
        assert torch.equal(y, c)
