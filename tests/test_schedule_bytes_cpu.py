"""What a decode schedule says it reads and what it allocates: those of its own cache format."""
import pytest
import torch

from long_context_emitting_b200 import api
from long_context_emitting_b200.schedule import DecodeSchedule, PagedQ4DecodeSchedule


@pytest.mark.parametrize("lens", [(4096, 0, 700), (1,)])
def test_bytes_and_workspace(monkeypatch, lens):
    made = []
    real = api.workspace
    monkeypatch.setattr(api, "workspace", lambda n, device: made.append(n) or real(n, device))
    B, Hq, Hkv = len(lens), 32, 8
    ks = [api.k_for_len(T) for T in lens]
    wide = DecodeSchedule(B, Hq, Hkv, lens, (0,), 2, "cpu")
    assert made == [max(api.decode_anchor_workspace_bytes(B, Hq, Hkv, max(lens)),
                        api.decode_reuse_workspace_bytes(B, Hq, Hkv, max(ks)))]
    assert wide.kv_bytes_per_layer == sum(lens) * Hkv * 512 and wide.reuse_bytes_per_layer == sum(ks) * Hkv * 512
    del made[:]
    q4 = PagedQ4DecodeSchedule(B, Hq, Hkv, lens, (0,), 2, "cpu", torch.zeros(64))
    assert made == [api.decode_anchor_paged_q4_workspace_bytes(B, Hq, Hkv, max(lens))]
    assert q4.ws.numel() == max(16, made[0])
    assert q4.kv_bytes_per_layer == sum(lens) * Hkv * 160 and q4.reuse_bytes_per_layer == sum(ks) * Hkv * 160
