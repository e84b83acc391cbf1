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


class Guarded:
    """A buffer in the middle of a larger one whose other bytes are known."""

    def __init__(self, shape, dtype, margin=4096):
        n = torch.Size(shape).numel() * dtype.itemsize
        self.all = torch.full((n + 2 * margin,), 0x5A, dtype=torch.uint8, device="cuda")
        self.inner = self.all[margin:margin + n].view(dtype).view(shape)
        self.margin = margin

    def untouched(self):
        return bool((self.all[:self.margin] == 0x5A).all() and (self.all[-self.margin:] == 0x5A).all())


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("tables", ["starts", "lens", "pages"])
def test_bad_tables_write_nothing_outside_the_buffers(bsfp, mode, tables):
    cache, batch, q = build(bsfp, mode, [200, 40, 100], [1, 12, 7], 4, 2, 64, 16, seed=4)
    T = q.shape[0]
    changes = {
        "starts": [dict(q_starts=i32(s)) for s in ([0, 900, 2, 3], [-5, 1, 2, T], [0, 1, 0, 3], [T, 2, 1, 0],
                                                  [0, 1, 2, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1, 0, T])],
        "lens": [dict(kv_lens=i32(n)) for n in ([2 ** 31 - 1, 5, 1], [-3, -2 ** 31, 100], [10 ** 6, 209, 0])],
        "pages": [dict(block_table=torch.full_like(batch.block_table, p)) for p in (-1, -2 ** 31, 2 ** 31 - 1,
                                                                                   cache.pages)]}[tables]
    for change in changes:
        bad = bsfp.KvBatch(batch.block_table, batch.kv_lens, batch.q_starts)
        for name, t in change.items():
            setattr(bad, name, t)
        for max_q in (1, T):
            for window in (0, 33):
                out, lse = Guarded((T, 4, 64), torch.bfloat16), Guarded((T, 4), torch.float32)
                ws = Guarded((bsfp.kv_attention_workspace_bytes(max_q, 4, 2, 64, 3),), torch.uint8)
                bsfp.kv_attention(q, cache, bad, max_q=max_q, window=window, out=out.inner, lse=lse.inner,
                                  workspace=ws.inner)
                assert out.untouched() and lse.untouched() and ws.untouched(), (change, max_q, window)


def test_append_writes_nothing_outside_the_cache(bsfp):
    from block_scaled_bit_fp_amd.kv import KvCache
    P, Hk, D, pages = 16, 3, 64, 4
    rows = pages * Hk * P
    parts = [(Guarded((rows, 8), torch.int32), Guarded((rows, 4), torch.uint8)) for _ in range(2)]
    k, v = (bsfp.QuantizedTensor(NVFP4, rows, D, c.inner, s.inner) for c, s in parts)
    cache = KvCache(k, v, Hk, P)
    x = torch.randn((12, Hk, D), device="cuda").to(torch.bfloat16)
    slots = torch.tensor([-1, -2 ** 63, 2 ** 63 - 1, pages * P, pages * P + 1, 2 ** 31, 2 ** 32, -17, 0, pages * P - 1,
                          5, 1 << 40], device="cuda")
    bsfp.kv_append(cache, x, x, slots)
    assert all(g.untouched() for pair in parts for g in pair)
    whole = bsfp.quantize(x[8:11].reshape(-1, D), NVFP4, global_scale="none")
    at = torch.tensor([((s // P * Hk) + h) * P + s % P for s in (0, pages * P - 1, 5) for h in range(Hk)], device="cuda")
    assert torch.equal(k.codes[at], whole.codes) and torch.equal(v.scales[at], whole.scales)
    left = torch.ones(rows, dtype=torch.bool, device="cuda")
    left[at] = False
    assert (k.codes[left] == 0x5A5A5A5A).all() and (v.scales[left] == 0x5A).all()
