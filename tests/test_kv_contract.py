"""Host-side checks of the paged cache's contract (no GPU needed, no kernel is launched): calls that a kernel
could not answer rightly come back as a status and a message."""
import ctypes as C

import pytest
import torch

ARG, UNSUPPORTED = 1, 2
R, P, M, F, T = 300, 16, 4, 50, 500

# Addresses of kv_plan's buffers, each with room for its own; never dereferenced.
NAMES = ("past", "q", "table", "free", "begin", "kv", "starts", "slots", "pos", "state")
SIZES = dict(past=4 * R, q=4 * R, table=4 * R * M, free=4 * F, begin=4, kv=4 * R, starts=4 * (R + 1), slots=8 * T,
             pos=4 * T, state=8)
AT = {n: (i + 1) << 16 for i, n in enumerate(NAMES)}
INPUTS, OUTPUTS = ("past", "q", "free", "begin"), ("table", "kv", "starts", "slots", "pos", "state")


@pytest.fixture(scope="module")
def b():
    import block_scaled_bit_fp_amd as b
    return b


def plan(b, **at):
    a = dict(AT, **at)
    status = b.lib().bsfp_kv_plan(a["past"], a["q"], R, P, a["table"], M, a["free"], F, a["begin"], T, a["kv"],
                                  a["starts"], a["slots"], a["pos"], a["state"], None)
    return status, b.lib().bsfp_last_error().decode()


@pytest.mark.parametrize("out", OUTPUTS)
@pytest.mark.parametrize("other", INPUTS + OUTPUTS)
def test_plan_refuses_buffers_that_overlap(b, out, other):
    """kv_plan(batch.kv_lens, ..., out=batch) above all: every workgroup reads the lengths that one writes."""
    if out == other:
        return
    for at in (AT[other], AT[other] + SIZES[other] - 4, AT[other] - SIZES[out] + 4):
        status, message = plan(b, **{out: at})
        assert status == ARG and "overlaps" in message, (at - AT[other], status, message)


@pytest.mark.parametrize("name", NAMES)
def test_plan_names_the_null_buffer(b, name):
    status, message = plan(b, **{name: None})
    assert status == ARG and "null" in message


def test_cache_descriptor_follows_its_fields(b):
    c = b.empty_kv_cache(b.MXFP4, 4, 2, 64, page_size=32, device="cpu")

    def fields():
        d = c.desc()._obj
        return d.pages, d.kv_heads, d.page_size, d.k.contents.codes, d.v.contents.codes
    at = c.k.codes.data_ptr(), c.v.codes.data_ptr()
    assert fields() == (4, 2, 32, *at)
    kept = c.desc()
    assert c.desc() is kept  # rebuilt only when something changed
    c.page_size = 64
    assert fields() == (2, 2, 64, *at)
    c.kv_heads = 1
    assert fields() == (4, 1, 64, *at)
    c.k.codes = c.k.codes.clone()
    assert fields() == (4, 1, 64, c.k.codes.data_ptr(), at[1])
    c.v = b.empty_quantized(b.MXFP4, c.k.rows, 64, "cpu")
    assert fields() == (4, 1, 64, c.k.codes.data_ptr(), c.v.codes.data_ptr())
