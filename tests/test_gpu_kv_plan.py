"""kv_plan from step to step: what a request has in the cache is carried over, also where it was refused."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from test_gpu_kv import NVFP4, i32, new_cache, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [0, 1, 7, 256, 257, 1500])
@pytest.mark.parametrize("short", [0, 5])
def test_next_lens(bsfp, R, short):
    """past + q of an admitted request, past of a refused one, and the other outputs as without it."""
    rng, P = np.random.default_rng([R, short]), 16
    past, q = rng.integers(0, 200, R), rng.integers(0, 40, R)
    if R > 5:
        past[1], q[3] = -4, -2  # lengths that refuse a request
    M = 20
    table = np.arange(R * M, dtype=np.int32).reshape(R, M)
    need = sum(max(0, -(-(p + n) // P) - -(-p // P)) for p, n in zip(past, q) if p >= 0 and n >= 0)
    free = np.arange(R * M, R * M + max(need - short, 0), dtype=np.int32)
    tokens = int(np.maximum(q, 0).sum())
    want = ref.plan(past, q, table, free, 0, tokens, P)
    got = bsfp.kv_plan(i32(past), i32(q), i32(table), i32(free), i32([0]), tokens=tokens, page_size=P)
    for name, w in zip(("block_table", "kv_lens", "q_starts", "slots", "positions", "state"), want):
        assert np.array_equal(getattr(got, name).cpu().numpy(), w), name
    # kv_lens is 0 where the request was refused, or where it has and gets nothing
    assert np.array_equal(got.next_lens.cpu().numpy(), np.where(want[1] > 0, past + q, past))


def test_out_of_an_older_batch_gets_next_lens(bsfp):
    past, q, table = i32([3]), i32([2]), i32([[0]])
    first = bsfp.kv_plan(past, q, table, i32([]), i32([0]), tokens=2, page_size=16)
    first.next_lens = None
    again = bsfp.kv_plan(past, q, table, i32([]), i32([0]), tokens=2, page_size=16, out=first)
    assert again is first and again.next_lens.tolist() == [5]


def test_a_refused_request_goes_on_where_it_stood(bsfp):
    """Three requests decode; one finds no page for a while.  Its keys, pages and later tokens are those of a
    run that had pages all along."""
    R, Hk, H, D, P, steps, gap = 3, 2, 4, 64, 16, 24, range(16, 20)
    rows = [(rand((R, Hk, D), 10 * i), rand((R, Hk, D), 10 * i + 1), rand((R, H, D), 10 * i + 2)) for i in range(steps)]
    cache = new_cache(bsfp, NVFP4, 12, Hk, D, P)
    past, table, begin = i32([0] * R), i32(np.full((R, 4), -1)), i32([0])
    plenty, scarce = i32(np.arange(12)), i32(np.arange(3))
    fed = [0] * R  # tokens that each request has had
    for i in range(steps + len(gap)):
        # in the gap the free list is used up and every request stands at a page's end
        free = scarce if i in gap else plenty
        k, v, q = (torch.stack([rows[min(fed[r], steps - 1)][x][r] for r in range(R)]) for x in range(3))
        batch = bsfp.kv_plan(past, i32([1] * R), table, free, begin, tokens=R, page_size=P)
        bsfp.kv_append(cache, k, v, batch.slots)
        out = bsfp.kv_attention(q, cache, batch, max_q=1)
        refused = int(batch.state[1])
        assert refused == (R if i in gap else 0)
        if refused:
            assert not out.any() and past.tolist() == [16] * R
        else:
            fed = [n + 1 for n in fed]
        past.copy_(batch.next_lens)
        begin.copy_(batch.state[:1])
        assert past.tolist() == fed
    # the same tokens without a gap
    whole = new_cache(bsfp, NVFP4, 12, Hk, D, P)
    t2 = i32(np.arange(12).reshape(3, 4))
    t = torch.arange(steps, device="cuda")
    for r in range(R):
        slots = t2[r, t // P].long() * P + t % P
        bsfp.kv_append(whole, torch.stack([x[0][r] for x in rows]), torch.stack([x[1][r] for x in rows]), slots)
    want = bsfp.kv_attention(rows[-1][2], whole, bsfp.KvBatch(t2, past, i32(np.arange(R + 1))), max_q=1)
    assert torch.equal(out, want)
