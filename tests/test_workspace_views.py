"""Workspaces that are views, without a GPU: a call writes from the view's first byte on."""
import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af

CPU = torch.device("cpu")


@pytest.fixture(autouse=True)
def _any_device(monkeypatch):
    monkeypatch.setattr(af, "_need", lambda *a, **k: None)


def test_views_with_less_memory_than_elements_are_not_taken():
    one = torch.zeros(16, dtype=torch.uint8)
    for ws in (one[:1].expand(4096), one.view(1, 16).expand(300, 16), one[3:4].expand(64)):
        got = af._workspace(64, CPU, ws)
        assert got.untyped_storage().data_ptr() != one.untyped_storage().data_ptr() and got.numel() == 64
        with pytest.raises(ValueError, match="ROPE_REUSE_TABLE"):
            af._workspace(64, CPU, ws, reuse_table=True)


def test_views_with_enough_memory_are():
    big = torch.zeros(4096, dtype=torch.uint8)
    for ws in (big, big[::2], big[96:], big.view(64, 64).t(), big[1024:].view(torch.float32)):
        assert af._workspace(1024, CPU, ws) is ws
    assert af._workspace(0, CPU, big) is None
