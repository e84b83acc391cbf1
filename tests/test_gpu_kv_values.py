"""kv_attention where values are extreme: logits of 1e5 and more.  Against fp64 over the values that the cache
stands for, with the tolerances of kv_reference.py."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from test_gpu_kv import MODES, NVFP4, build, new_cache, rand

pytestmark = pytest.mark.gpu


# Decode, drafts, prompts, and one request whose keys are cut into parts.
LAYOUTS = [pytest.param([200, 90], [1, 1], id="decode"), pytest.param([200, 61], [4, 3], id="drafts"),
           pytest.param([260, 200], [70, 40], id="prompt"), pytest.param([2100], [1], id="decode-parts"),
           pytest.param([1500], [9], id="prompt-parts")]


def stairs(bsfp, mode, kv, q_lens, logit, step, down):
    """Logits near `logit` that rise (or fall) key by key in steps of `step` log2 units: the first 64 columns
    give the height, the others, ones and zeros, the step."""
    heads, kv_heads, D, P = 4, 2, 128, 64
    cache, batch, q = build(bsfp, mode, kv, q_lens, heads, kv_heads, D, P, seed=int(logit) % 1000)
    if mode == NVFP4:
        cache = new_cache(bsfp, mode, cache.pages, kv_heads, D, P, scaled=False)
    for r, n in enumerate(kv):
        t = torch.arange(n, device="cuda")
        slots = batch.block_table[r, t // P].long() * P + t % P
        up = (n - 1 - t if down else t) * 64 // n
        k = torch.full((n, kv_heads, D), 4.0, device="cuda")
        k[..., 64:] = (torch.arange(64, device="cuda") < up[:, None, None]).float()
        bsfp.kv_append(cache, k.to(torch.bfloat16), rand((n, kv_heads, D), 70 + r), slots)
    scale = 1.0 / np.sqrt(D)
    q = torch.full_like(q, logit / scale / 256)
    q[..., 64:] = step / (scale * 1.4426950408889634)
    return cache, batch, q


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("kv,q_lens", LAYOUTS)
@pytest.mark.parametrize("logit", [1e5, -1e5, 1e6, 1e7, 1e12])
def test_large_finite_logits_stay_finite(bsfp, mode, kv, q_lens, logit):
    for step, down in ((0.97, False), (0.5, False), (1.7, False), (0.97, True)):
        cache, batch, q = stairs(bsfp, mode, kv, q_lens, logit, step, down)
        out, lse = bsfp.kv_attention(q, cache, batch, return_lse=True)
        wout, wlse, otol, ltol = ref.attention(q, cache, batch.block_table, batch.kv_lens, batch.q_starts,
                                               float(np.float32(1.0 / np.sqrt(128))))
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.isfinite(out).all() and np.isfinite(lse).all(), (step, down)
        assert (np.abs(lse - wlse) <= ltol).all()
        assert (np.abs(out - wout) <= otol).all()
        # where that tolerance says little: a mean of values, and no larger than the largest of them
        assert np.abs(out).max() < 8.0
