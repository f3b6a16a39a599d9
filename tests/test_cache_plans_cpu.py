"""What is kept of a call's shapes holds for the device that it was found on:
the attention's workspace goes by the number of its multiprocessors."""
import types

import pytest
import torch

import rejection_sampling_verify_b200 as psi
from rejection_sampling_verify_b200 import cache


@pytest.mark.parametrize("out", [False, True])
def test_workspace_follows_the_device(monkeypatch, out):
    current = [0]
    monkeypatch.setattr(cache, "_on_device", lambda ref, named: current[0])
    monkeypatch.setattr(cache, "_new_status", lambda dev: torch.zeros(1, dtype=torch.int32))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(cache, "psi_attend_block_workspace_bytes",
                        lambda *a: 256 * (1 + current[0]))
    given = []
    monkeypatch.setattr(cache, "psi_attend_block", lambda *a: given.append(a[-2]) or psi.PSI_OK)
    monkeypatch.setattr(cache, "_binding", types.SimpleNamespace(attend=lambda *a: None))
    monkeypatch.setattr(cache, "_plans", {})
    q = torch.ones(2, 3, 4, 64).bfloat16()
    pool = torch.ones(8, 16, 2, 64).bfloat16()
    table, lens = torch.ones(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    res = psi.AttendResult(q.clone(), None, lens[:1].clone()) if out else None
    for current[0] in (0, 1, 1, 0):
        psi.attend_block(q, pool, pool, table, lens, out=res)
    assert given == [256, 512, 512, 256]
