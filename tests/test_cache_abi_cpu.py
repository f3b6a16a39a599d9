"""CPU checks of the cache's entry points: every argument error is returned
before anything is launched, and the binding refuses tensors that do not
match what the kernels read and write."""
import math

import pytest
import torch

import rejection_sampling_verify_b200 as psi

FAKE = 0x10000  # a 64 KB-aligned fake device address: never dereferenced


def _layout(**over):
    f = dict(dtype=psi.PSI_DTYPE_BF16, layers=1, num_pages=8, page_size=16, kv_heads=2,
             head_dim=64, layer_stride=8 * 2048, page_stride=2048, slot_stride=128, head_stride=64)
    f.update(over)
    return psi.CacheLayout(*f.values())


BAD_LAYOUTS = [
    (dict(dtype=5), psi.PSI_ERR_INVALID_ARG),
    (dict(layers=0), psi.PSI_ERR_INVALID_ARG),
    (dict(num_pages=0), psi.PSI_ERR_INVALID_ARG),
    (dict(page_size=0), psi.PSI_ERR_INVALID_ARG),
    (dict(page_size=1025), psi.PSI_ERR_INVALID_ARG),
    (dict(kv_heads=0), psi.PSI_ERR_INVALID_ARG),
    (dict(head_dim=0), psi.PSI_ERR_INVALID_ARG),
    (dict(head_dim=60), psi.PSI_ERR_UNSUPPORTED),
    (dict(head_dim=264, head_stride=264, slot_stride=528, page_stride=8448),
     psi.PSI_ERR_UNSUPPORTED),
    (dict(slot_stride=-128), psi.PSI_ERR_INVALID_ARG),
    (dict(slot_stride=132), psi.PSI_ERR_MISALIGNED),
    (dict(head_stride=56), psi.PSI_ERR_INVALID_ARG),
    (dict(page_stride=0), psi.PSI_ERR_INVALID_ARG),
]


def _append(layout=None, **over):
    a = dict(k_pages=FAKE, v_pages=FAKE, page_table=FAKE, max_pages=4, lens=FAKE, N=2, R=3,
             q_heads=4, q=FAKE, q_row_stride=512, q_head_stride=64, k=FAKE, k_row_stride=512,
             k_head_stride=64, v=FAKE, v_row_stride=512, v_head_stride=64, q_weight=FAKE,
             k_weight=FAKE, eps=1e-6, inv_freq=FAKE, rotary_dim=64, interleaved=0, rope_scale=1.0,
             parents=None, out_q=FAKE, dev_status=None, stream=None)
    a.update(over)
    return psi.psi_cache_append(layout or _layout(), **a)


def _attend(layout=None, **over):
    a = dict(k_pages=FAKE, v_pages=FAKE, page_table=FAKE, max_pages=4, lens=FAKE, N=2, R=3,
             q_heads=4, q=FAKE, q_row_stride=512, q_head_stride=64, parents=None, scale=0.1,
             out_o=FAKE, out_lse=None, dev_status=None, workspace=FAKE, workspace_bytes=1 << 30,
             stream=None)
    a.update(over)
    return psi.psi_attend_block(layout or _layout(), **a)


def _commit(layout=None, **over):
    a = dict(k_pages=FAKE, v_pages=FAKE, page_table=FAKE, max_pages=4, lens=FAKE, N=2, M=8,
             path_nodes=FAKE, path_len=FAKE, out_lens=2 * FAKE, dev_status=None, stream=None)
    a.update(over)
    return psi.psi_cache_commit(layout or _layout(), **a)


def _state(**over):
    f = dict(page_table=FAKE, page_counts=FAKE, refs=FAKE, free_pages=FAKE, n_free=FAKE)
    f.update(over)
    return psi.PageStatePtrs(*f.values())


def _fork(layout=None, **over):
    a = dict(k_pages=FAKE, v_pages=FAKE, N=4, max_pages=4, lens=FAKE, out_lens=FAKE,
             in_state=_state(), out_state=_state(), K=2, src=FAKE, dst=FAKE, dev_status=None,
             workspace=FAKE, workspace_bytes=1 << 20, stream=None)
    a.update(over)
    return psi.psi_cache_fork(layout or _layout(), **a)


@pytest.mark.parametrize("call", [_append, _attend, _commit, _fork])
@pytest.mark.parametrize("over,want", BAD_LAYOUTS)
def test_bad_layouts_are_refused(call, over, want):
    assert call(_layout(**over)) == want
    assert psi.psi_last_error()


@pytest.mark.parametrize("call", [_append, _attend, _commit])
@pytest.mark.parametrize("over,want", [
    (dict(k_pages=None), psi.PSI_ERR_INVALID_ARG),
    (dict(page_table=None), psi.PSI_ERR_INVALID_ARG),
    (dict(lens=None), psi.PSI_ERR_INVALID_ARG),
    (dict(max_pages=0), psi.PSI_ERR_INVALID_ARG),
    (dict(max_pages=1 << 28), psi.PSI_ERR_INVALID_ARG),
    (dict(N=0), psi.PSI_ERR_INVALID_ARG),
    (dict(k_pages=FAKE + 8), psi.PSI_ERR_MISALIGNED),
    (dict(lens=FAKE + 2), psi.PSI_ERR_MISALIGNED),
])
def test_bad_tables_are_refused(call, over, want):
    assert call(**over) == want


@pytest.mark.parametrize("over,want", [
    (dict(R=0), psi.PSI_ERR_INVALID_ARG),
    (dict(R=psi.PSI_MAX_BLOCK_ROWS + 1), psi.PSI_ERR_INVALID_ARG),
    (dict(q_heads=3), psi.PSI_ERR_INVALID_ARG),
    (dict(q_heads=0), psi.PSI_ERR_INVALID_ARG),
    (dict(q=None), psi.PSI_ERR_INVALID_ARG),
    (dict(q=FAKE + 8), psi.PSI_ERR_MISALIGNED),
    (dict(q_row_stride=516), psi.PSI_ERR_MISALIGNED),
    (dict(q_head_stride=32), psi.PSI_ERR_INVALID_ARG),
])
@pytest.mark.parametrize("call", [_append, _attend])
def test_bad_queries_are_refused(call, over, want):
    assert call(**over) == want


@pytest.mark.parametrize("over,want", [
    (dict(rotary_dim=63), psi.PSI_ERR_INVALID_ARG),
    (dict(rotary_dim=66), psi.PSI_ERR_INVALID_ARG),
    (dict(rotary_dim=-2), psi.PSI_ERR_INVALID_ARG),
    (dict(inv_freq=None), psi.PSI_ERR_INVALID_ARG),
    (dict(inv_freq=FAKE + 4), psi.PSI_ERR_MISALIGNED),
    (dict(eps=-1.0), psi.PSI_ERR_INVALID_ARG),
    (dict(eps=math.nan), psi.PSI_ERR_INVALID_ARG),
    (dict(rope_scale=math.inf), psi.PSI_ERR_INVALID_ARG),
    (dict(out_q=None), psi.PSI_ERR_INVALID_ARG),
    (dict(v=None), psi.PSI_ERR_INVALID_ARG),
    (dict(k_weight=FAKE + 2), psi.PSI_ERR_MISALIGNED),
])
def test_append_refuses(over, want):
    assert _append(**over) == want


@pytest.mark.parametrize("over,want", [
    (dict(out_o=None), psi.PSI_ERR_INVALID_ARG),
    (dict(scale=math.nan), psi.PSI_ERR_INVALID_ARG),
    (dict(out_lse=FAKE + 2), psi.PSI_ERR_MISALIGNED),
    (dict(workspace=None), psi.PSI_ERR_WORKSPACE),
    (dict(workspace_bytes=0), psi.PSI_ERR_WORKSPACE),
])
def test_attend_refuses(over, want):
    assert _attend(**over) == want


@pytest.mark.parametrize("over,want", [
    (dict(M=0), psi.PSI_ERR_INVALID_ARG),
    (dict(M=psi.PSI_MAX_BLOCK_ROWS), psi.PSI_ERR_INVALID_ARG),
    (dict(path_nodes=None), psi.PSI_ERR_INVALID_ARG),
    (dict(out_lens=FAKE), psi.PSI_ERR_INVALID_ARG),      # the lengths themselves
    (dict(out_lens=FAKE + 4), psi.PSI_ERR_INVALID_ARG),  # overlapping them
    (dict(path_len=FAKE + 1), psi.PSI_ERR_MISALIGNED),
])
def test_commit_refuses(over, want):
    assert _commit(**over) == want


@pytest.mark.parametrize("over,want", [
    (dict(K=0), psi.PSI_ERR_INVALID_ARG),
    (dict(K=5), psi.PSI_ERR_INVALID_ARG),
    (dict(src=None), psi.PSI_ERR_INVALID_ARG),
    (dict(in_state=None), psi.PSI_ERR_INVALID_ARG),
    (dict(out_state=_state(refs=None)), psi.PSI_ERR_INVALID_ARG),
    (dict(in_state=_state(free_pages=FAKE + 2)), psi.PSI_ERR_MISALIGNED),
    (dict(workspace=None), psi.PSI_ERR_WORKSPACE),
    (dict(workspace_bytes=4), psi.PSI_ERR_WORKSPACE),
])
def test_fork_refuses(over, want):
    assert _fork(**over) == want


@pytest.mark.parametrize("over,want", [
    (dict(N=0), psi.PSI_ERR_INVALID_ARG),
    (dict(page_size=0), psi.PSI_ERR_INVALID_ARG),
    (dict(extra=-1), psi.PSI_ERR_INVALID_ARG),
    (dict(lens=None), psi.PSI_ERR_INVALID_ARG),
    (dict(out_state=None), psi.PSI_ERR_INVALID_ARG),
    (dict(in_state=_state(n_free=FAKE + 1)), psi.PSI_ERR_MISALIGNED),
])
def test_resize_refuses(over, want):
    a = dict(N=4, max_pages=4, num_pages=8, page_size=16, lens=FAKE, extra=0, in_state=_state(),
             out_state=_state(), dev_status=None, stream=None)
    a.update(over)
    assert psi.psi_cache_resize(**a) == want


def test_workspace_queries():
    lay = _layout()
    assert psi.psi_attend_block_workspace_bytes(lay, 2, 3, 4, 4) % 256 == 0
    assert psi.psi_attend_block_workspace_bytes(lay, 2, 3, 4, 4) > 0
    assert psi.psi_attend_block_workspace_bytes(lay, 0, 3, 4, 4) == 0
    assert psi.psi_attend_block_workspace_bytes(lay, 2, 3, 3, 4) == 0
    assert psi.psi_attend_block_workspace_bytes(_layout(head_dim=60), 2, 3, 4, 4) == 0
    assert psi.psi_cache_fork_workspace_bytes(0) == 0
    assert psi.psi_cache_fork_workspace_bytes(3) >= 36


def _tensors(N=2, R=3, Hq=4, H=2, D=64, S=16, P=8, dt=torch.bfloat16):
    return dict(q=torch.zeros(N, R, Hq, D, dtype=dt), kp=torch.zeros(P, S, H, D, dtype=dt),
                vp=torch.zeros(P, S, H, D, dtype=dt), k=torch.zeros(N, R, H, D, dtype=dt),
                table=torch.zeros(N, 4, dtype=torch.int32),
                lens=torch.zeros(N, dtype=torch.int32))


def test_binding_refuses_what_the_kernels_cannot_read():
    t = _tensors()
    ok = (t["q"], t["kp"], t["vp"], t["table"], t["lens"])
    with pytest.raises(ValueError, match="CUDA"):  # well-formed tensors reach the device check
        psi.attend_block(*ok)

    def attend(**over):
        u = dict(t, **over)
        return psi.attend_block(u["q"], u["kp"], u["vp"], u["table"], u["lens"],
                                parents=u.get("parents"))

    for over, match in [
            (dict(lens=t["lens"].long()), "lens"), (dict(lens=t["lens"][:1]), "lens"),
            (dict(table=t["table"].long()), "page_table"), (dict(table=t["table"][:1]), "page_table"),
            (dict(vp=t["vp"].float()), "dtype"), (dict(vp=t["vp"].transpose(1, 2)), "shape"),
            (dict(q=t["q"].float()), "q must"), (dict(q=t["q"][..., :32]), "q must"),
            (dict(q=t["q"].transpose(0, 1).contiguous().transpose(0, 1)), "evenly"),
            (dict(parents=torch.zeros(2, 3, dtype=torch.int32)), "parents")]:
        with pytest.raises(ValueError, match=match):
            attend(**over)
    with pytest.raises(ValueError, match="out.o"):
        psi.attend_block(*ok, out=psi.AttendResult(t["q"][:1], None, t["lens"][:1]))
    with pytest.raises(ValueError, match="inv_freq"):
        psi.cache_append(t["q"], t["k"], t["k"], *ok[1:], inv_freq=torch.ones(32))
    with pytest.raises(ValueError, match="q_weight"):
        psi.cache_append(t["q"], t["k"], t["k"], *ok[1:], q_weight=torch.ones(64))
    with pytest.raises(ValueError, match="CUDA"):
        psi.cache_append(t["q"], t["k"], t["k"], *ok[1:])
    lk = t["kp"][None]
    path, n = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        psi.cache_commit(lk, lk, t["table"], t["lens"], path, n)
    with pytest.raises(ValueError, match="path_len"):
        psi.cache_commit(lk, lk, t["table"], t["lens"], path, n[:1])
    with pytest.raises(ValueError, match="dims"):
        psi.cache_commit(t["kp"], t["kp"], t["table"], t["lens"], path, n)
    pages = psi.PageState.empty(2, 4, 8, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        psi.cache_resize(pages, t["lens"], 0, 16)
    with pytest.raises(ValueError, match="CUDA"):
        psi.cache_fork(lk, lk, pages, t["lens"], n, n)
    pages.free = pages.free[:7]
    with pytest.raises(ValueError, match="free"):
        psi.cache_resize(pages, t["lens"], 0, 16)
    with pytest.raises(ValueError, match="free"):
        psi.cache_fork(lk, lk, pages, t["lens"], n, n)


def test_rope_frequencies():
    inv, scale = psi.rope_frequencies(128, 1e4, device="cpu")
    assert inv.dtype == torch.float64 and scale == 1.0
    assert torch.allclose(inv, 1e4 ** (-torch.arange(64, dtype=torch.float64) / 64))
    lin, _ = psi.rope_frequencies(128, 1e4, 4.0, "linear", device="cpu")
    assert torch.equal(lin, inv / 4)
    # the shortest wavelength is kept, the longest stretched by the factor
    ntk, _ = psi.rope_frequencies(128, 1e4, 4.0, "ntk", device="cpu")
    assert ntk[0] == 1 and abs(float(ntk[-1] * 4 / inv[-1]) - 1) < 1e-12
    yarn, ys = psi.rope_frequencies(128, 1e4, 4.0, "yarn", 4096, device="cpu")
    turns = 4096 * inv / (2 * math.pi)
    assert torch.equal(yarn[turns > 33], inv[turns > 33])
    assert torch.allclose(yarn[turns < 0.9], inv[turns < 0.9] / 4, rtol=1e-12)
    assert bool((yarn <= inv).all()) and bool((yarn >= inv / 4).all())
    assert abs(ys - (0.1 * math.log(4.0) + 1)) < 1e-15
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, factor=0.5),
                dict(rotary_dim=8, scaling="other")):
        with pytest.raises(ValueError):
            psi.rope_frequencies(device="cpu", **bad)
