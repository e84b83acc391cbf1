"""kv_attention's buffers: the workspace that a call needs, and nothing written outside out, lse and workspace
whatever the tables hold."""
import pytest
import torch

from test_gpu_kv import MODES, NVFP4, build, i32

pytestmark = pytest.mark.gpu


def test_workspace_of_a_decode_step(bsfp):
    """One new token a request needs no partial states of prompts, however many requests there are."""
    kv = [3000, 70, 1, 0] * 10
    cache, batch, q = build(bsfp, NVFP4, kv, [1] * 40, 8, 1, 128, 64, seed=2)
    want = bsfp.kv_attention(q, cache, batch, return_lse=True)
    ws = bsfp.kv_attention_workspace(40, 8, cache, 40, max_q=1)
    assert ws.numel() == bsfp.kv_attention_workspace_bytes(1, 8, 1, 128, 40)
    assert 2 * ws.numel() < bsfp.kv_attention_workspace(40, 8, cache, 40).numel()
    assert bsfp.kv_attention_workspace(40, 8, cache, 40, max_q=1000).numel() == \
        bsfp.kv_attention_workspace(40, 8, cache, 40).numel()
    out, lse = bsfp.kv_attention(q, cache, batch, max_q=1, workspace=ws, return_lse=True)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for args in (dict(), dict(max_q=3)):  # 24 rows per kv head may be a prompt's
        with pytest.raises(bsfp.BsfpError) as ei:
            bsfp.kv_attention(q, cache, batch, workspace=ws, **args)
        assert ei.value.status == 1
    with pytest.raises(bsfp.BsfpError):
        bsfp.kv_attention(q, cache, batch, max_q=1, workspace=ws[:-16])
