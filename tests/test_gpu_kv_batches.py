"""Large mixed batches: more requests than lanes beside prompts, more rows than a launch of kv_append holds at
once, and steps that begin at page ends."""
import numpy as np
import pytest
import torch

from test_gpu_kv import MODES, NVFP4, build, cache_rows, check_attention, check_plan, new_cache, rand

pytestmark = pytest.mark.gpu


def mixed(rng, R, prompts):
    """(kv, q_lens): one new token for most, none or no key for some, 5 to 40 for `prompts` of them."""
    kv = rng.integers(0, 70, R)
    q = np.ones(R, np.int64)
    q[rng.random(R) < 0.1] = 0
    kv[rng.random(R) < 0.1] = 0
    at = rng.permutation(R)[:prompts]
    q[at] = rng.integers(5, 41, prompts)
    kv[at] = q[at] + rng.integers(-3, 50, prompts)
    return [int(max(x, 0)) for x in kv], [int(x) for x in q]


@pytest.mark.parametrize("R,prompts", [(63, 5), (64, 64), (65, 9), (130, 20), (130, 1), (700, 25)])
@pytest.mark.parametrize("window", [0, 9])
@pytest.mark.parametrize("mode", MODES)
def test_prompts_among_many_requests(bsfp, R, prompts, window, mode):
    kv, q_lens = mixed(np.random.default_rng([R, prompts]), R, prompts)
    cache, batch, q = build(bsfp, mode, kv, q_lens, 4, 1, 64, 16, seed=R, pad=3)
    check_attention(bsfp, cache, batch, q, window=window)


@pytest.mark.parametrize("where", [0, 64, 129])
def test_one_prompt_among_requests_of_nothing(bsfp, where):
    """All but one of 130 requests have no work for the prompt kernel; the one has parts."""
    kv, q_lens = [0] * 130, [1, 0] * 65
    kv[where], q_lens[where] = 1300, 30
    cache, batch, q = build(bsfp, NVFP4, kv, q_lens, 4, 1, 64, 16, seed=where)
    check_attention(bsfp, cache, batch, q, max_q=30)


@pytest.mark.parametrize("mode", MODES)
def test_append_of_more_rows_than_lanes(bsfp, mode):
    """The grid holds 16 workgroups of 256 words per CU: 8209 tokens of 8 x 128 go round twice, skipped ones
    among those of the second round."""
    T, Hk, D, P = 8209, 8, 128, 64
    pages = T // P + 2
    assert T * Hk * D // 8 > torch.cuda.get_device_properties(0).multi_processor_count * 16 * 256
    cache = new_cache(bsfp, mode, pages, Hk, D, P)
    k, v = rand((T, Hk, D), 1, 3.0), rand((T, Hk, D), 2)
    slots = torch.randperm(pages * P, device="cuda")[:T]
    skipped = torch.tensor([0, 8192, 8200, T - 1], device="cuda")
    slots[skipped] = -1
    for t in (cache.k, cache.v):
        t.codes.fill_(0x33333333)
    bsfp.kv_append(cache, k, v, slots)
    live = slots >= 0
    rows = cache_rows(slots[live], Hk, P).reshape(-1)
    left = torch.ones(cache.k.rows, dtype=torch.bool, device="cuda")
    left[rows] = False
    for t, x in ((cache.k, k), (cache.v, v)):
        want = bsfp.empty_quantized(mode, T * Hk, D, global_scale=False)
        want.global_scale = t.global_scale
        bsfp.quantize(x.view(-1, D), mode, global_scale="given" if t.global_scale is not None else "none", out=want)
        keep = live[:, None].expand(T, Hk).reshape(-1)
        assert torch.equal(t.codes[rows], want.codes[keep])
        assert torch.equal(t.scales[rows], want.scales[keep])
        assert t.biases is None or torch.equal(t.biases[rows], want.biases[keep])
        assert (t.codes[left] == 0x33333333).all()


@pytest.mark.parametrize("P", [16, 64, 256])
@pytest.mark.parametrize("R", [3, 64, 300])
def test_plan_of_steps_that_begin_at_page_ends(bsfp, P, R):
    rng = np.random.default_rng([P, R])
    past = rng.integers(0, 5, R) * P
    q = rng.choice([0, 1, P - 1, P, P + 1, 3 * P], R)
    M = int((past + q).max() // P + 1)
    old = past // P
    need = -(-(past + q) // P) - old
    ids = rng.permutation(int(old.sum() + need.sum())).astype(np.int32)
    table = np.full((R, M), -1, np.int32)
    at = 0
    for r in range(R):
        table[r, :old[r]] = ids[at:at + old[r]]
        at += old[r]
    check_plan(bsfp, past, q, table, ids[at:], 0, int(q.sum()), P)
    check_plan(bsfp, past, q, table, ids[at:], 3, int(q.sum()), P)  # three pages short
