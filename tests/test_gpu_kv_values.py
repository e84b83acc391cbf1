"""kv_attention where values are extreme: logits of 1e5 and more, values near the end of bf16's range, and
values that are not finite at keys that only some rows of a request see.  Against fp64 over the values that
the cache stands for, with the tolerances of kv_reference.py."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from test_gpu_kv import AFFINE, MODES, MXFP4, NVFP4, build, check_attention, new_cache, rand

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


def reach_of(batch, q_lens, r):
    """The position of the request's first new token."""
    return int(batch.kv_lens[r]) - q_lens[r]


@pytest.mark.parametrize("mode", [NVFP4, AFFINE])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv,q_lens,heads,window", [
    ([100, 61], [4, 7], 4, 0), ([100, 40], [16, 3], 1, 5), ([260, 200], [70, 40], 4, 0), ([300, 129], [129, 60], 1, 0),
    ([300, 129], [129, 60], 2, 20), ([2100], [5], 2, 0), ([1500], [12], 4, 0)])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(bsfp, mode, D, kv, q_lens, heads, window):
    """One key of the new tokens holds NaN and infinities in one group of its values: rows before it (or
    past its window) are those of a cache without it, rows that see it are not finite there."""
    P = 32
    cache, batch, q = build(bsfp, mode, kv, q_lens, heads, 1, D, P, seed=D + heads)
    clean = bsfp.kv_attention(q, cache, batch, window=window, return_lse=True)
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    G = 64 if mode == AFFINE else 16
    want = clean[0].clone()
    bad_rows = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    group = D // G - 1
    for r in range(len(kv)):
        t = reach_of(batch, q_lens, r) + q_lens[r] // 2  # seen by the later half of the rows
        row = int(batch.block_table[r, t // P]) * P + t % P
        if mode == AFFINE:
            cache.v.scales[row, group] = float("inf")
            cache.v.biases[row, group] = float("nan")
        else:
            cache.v.scales[row, group] = 0x7F
        pos = torch.arange(q_lens[r], device="cuda") + reach_of(batch, q_lens, r)
        sees = pos >= t
        if window:
            sees &= pos < t + window
        bad_rows[starts[r]:starts[r + 1]] = sees
    out, lse = bsfp.kv_attention(q, cache, batch, window=window, return_lse=True)
    assert torch.equal(lse, clean[1])
    cols = slice(group * G, group * G + G)
    assert torch.equal(out[~bad_rows], want[~bad_rows])
    assert torch.isnan(out[bad_rows][..., cols]).all()


def test_infinite_inputs_reach_only_the_rows_that_see_them(bsfp):
    """The same through kv_append: an affine row with an infinity has no finite scale."""
    for kv, q_lens in (([90], [5]), ([400], [150])):
        cache, batch, q = build(bsfp, AFFINE, kv, q_lens, 2, 1, 128, 64, seed=5)
        clean = bsfp.kv_attention(q, cache, batch)
        t = kv[0] - 2
        v = rand((1, 1, 128), 9)
        v[0, 0, 3] = float("inf")
        slot = batch.block_table[0, t // 64].long().view(1) * 64 + t % 64
        bsfp.kv_append(cache, rand((1, 1, 128), 10), v, slot)
        out = bsfp.kv_attention(q, cache, batch)
        assert torch.equal(out[:-2], clean[:-2])
        assert not torch.isfinite(out[-2:, :, :64]).any() and torch.isfinite(out[-2:, :, 64:]).all()


@pytest.mark.parametrize("mode", [MXFP4, AFFINE])
@pytest.mark.parametrize("kv,q_lens", LAYOUTS)
def test_values_near_the_end_of_the_range(bsfp, mode, kv, q_lens):
    """Means of values of 2^112 to 2^118 are finite."""
    cache, batch, q = build(bsfp, mode, kv, q_lens, 4, 2, 128, 64, seed=31)
    for r, n in enumerate(kv):
        t = torch.arange(n, device="cuda")
        slots = batch.block_table[r, t // 64].long() * 64 + t % 64
        v = (rand((n, 2, 128), 50 + r).float().clamp(-4, 4) * 2.0 ** 115).to(torch.bfloat16)
        bsfp.kv_append(cache, rand((n, 2, 128), 60 + r), v, slots)
    check_attention(bsfp, cache, batch, q)


def test_window_and_max_q_beyond_32_bits(bsfp):
    """No request is that long: as without a window, and as without a bound."""
    cache, batch, q = build(bsfp, NVFP4, [100, 80], [1, 30], 4, 1, 64, 16, seed=8)
    want = bsfp.kv_attention(q, cache, batch)
    for big in (2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63):
        assert torch.equal(bsfp.kv_attention(q, cache, batch, window=big), want), big
        assert torch.equal(bsfp.kv_attention(q, cache, batch, max_q=big + 1), want), big
    for bad in (dict(window=-2 ** 32), dict(max_q=-2 ** 32 + 1)):
        with pytest.raises(bsfp.BsfpError) as ei:
            bsfp.kv_attention(q, cache, batch, **bad)
        assert ei.value.status == 1


def put(bsfp, cache, batch, r, t, P, v):
    """The key t of request r: some K (the same each time) and the values v."""
    slot = batch.block_table[r, t // P].long().view(1) * P + t % P
    bsfp.kv_append(cache, rand(v.shape, t + 1), v, slot)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 30, 2.0 ** 60, 1e30, 3e38, float("inf")])
@pytest.mark.parametrize("kv,q_lens,heads,window", [
    ([100, 61], [4, 7], 4, 0), ([100, 40], [16, 3], 1, 5), ([12, 9], [12, 9], 1, 0), ([260, 200], [70, 40], 4, 0),
    ([300, 129], [129, 60], 1, 0), ([300, 129], [129, 60], 2, 20), ([400, 250], [200, 90], 1, 70), ([1500], [12], 4, 0),
    ([2100], [4], 4, 0)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_huge_values_reach_only_the_rows_that_see_them(bsfp, mode, size, kv, q_lens, heads, window, D):
    """Two new tokens, one of them a million times larger, with values far beyond the others': rows that do not
    see them are, within the tolerance, those over the values that they do see; to the rows that see them the
    huge ones come through."""
    P, scale = 32, float(np.float32(1.0 / np.sqrt(D)))
    cols = [7, D - 28]
    cache, batch, q = build(bsfp, mode, kv, q_lens, heads, 1, D, P, seed=heads + q_lens[0])
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    sees = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    huge = [(r, kv[r] - n + at, s) for r, n in enumerate(q_lens) for at, s in ((n // 3, size / 2 ** 20), (n // 2, size))]
    for r, t, s in huge:
        v = rand((1, 1, D), t)
        v[0, 0, cols] = s
        put(bsfp, cache, batch, r, t, P, v)
        pos = torch.arange(q_lens[r], device="cuda") + kv[r] - q_lens[r]
        sees[starts[r]:starts[r + 1]] |= (pos >= t) & (pos < t + window if window else pos >= t)
    out, lse = bsfp.kv_attention(q, cache, batch, window=window, return_lse=True)
    got, sees = out.double().cpu().numpy(), sees.cpu().numpy()
    assert not torch.isnan(lse).any() and not sees.all() and sees.any()
    if size <= 1e30:
        want, _, tol, _ = ref.attention(q, cache, batch.block_table, batch.kv_lens, batch.q_starts, scale, window)
        assert (np.abs(got - want)[sees][..., cols] <= tol[sees][..., cols]).all()
    # the reference over a cache in which those keys' values are small ones, and the same keys
    for r, t, _ in huge:
        put(bsfp, cache, batch, r, t, P, rand((1, 1, D), t))
    want, wlse, tol, ltol = ref.attention(q, cache, batch.block_table, batch.kv_lens, batch.q_starts, scale, window)
    err = np.abs(got - want)[~sees]
    assert (err <= tol[~sees]).all(), err.max()
    assert (np.abs(lse.double().cpu().numpy() - wlse) <= ltol).all()
