"""The binding's handle of the current stream where torch has no raw form of it (no GPU needed)."""

import importlib.util
import types

import torch


def test_public_form_where_torch_has_no_raw_one(monkeypatch):
    import gated_delta_rule_101_amd.block as block
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: types.SimpleNamespace(cuda_stream=100 + d))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    spec = importlib.util.spec_from_file_location("gated_delta_rule_101_amd.block_again", block.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    with again._on(torch.device("cuda", 3), None) as handle:
        assert handle == 103
