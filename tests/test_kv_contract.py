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


class Fake:
    """A tensor that is nowhere, named to stand on a device; its pointer must never be asked for."""

    def __init__(self, shape, dtype=torch.int32, device="cuda:0"):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self.is_cuda = self.device.type == "cuda"

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def stride(self):
        n = [1]
        for s in reversed(self.shape[1:]):
            n.insert(0, n[0] * s)
        return tuple(n)

    def is_contiguous(self):
        return True

    def new_empty(self, shape, dtype=None):
        return Fake((shape,) if isinstance(shape, int) else shape, dtype or self.dtype, self.device)

    def data_ptr(self):
        raise AssertionError("the call was not refused")


BF16 = torch.bfloat16


def fake_cache(b, device="cuda:0"):
    def side():
        return b.QuantizedTensor(b.MXFP4, 64, 64, Fake((64, 8), device=device), Fake((64, 2), torch.uint8, device))
    return b.KvCache(side(), side(), kv_heads=2, page_size=16)


def attention_call(b, **change):
    a = dict(q=Fake((3, 4, 64), BF16), table=Fake((2, 5)), lens=Fake((2,)), starts=Fake((3,)), cache=fake_cache(b),
             out=Fake((3, 4, 64), BF16), lse=Fake((3, 4), torch.float32), workspace=Fake((1 << 28,), torch.uint8))
    a.update(change)
    return b.kv_attention(a["q"], a["cache"], b.KvBatch(a["table"], a["lens"], a["starts"]), out=a["out"], lse=a["lse"],
                          workspace=a["workspace"])


@pytest.mark.parametrize("name,shape,dtype", [
    ("q", (3, 4, 64), BF16), ("table", (2, 5), torch.int32), ("lens", (2,), torch.int32), ("starts", (3,), torch.int32),
    ("out", (3, 4, 64), BF16), ("lse", (3, 4), torch.float32), ("workspace", (1 << 28,), torch.uint8)])
def test_attention_refuses_tensors_of_another_device(b, name, shape, dtype):
    with pytest.raises(ValueError, match="cuda"):
        attention_call(b, **{name: Fake(shape, dtype, "cuda:1")})


@pytest.mark.parametrize("device", ["cpu", "cuda:1"])
def test_calls_refuse_a_cache_of_another_device(b, device):
    with pytest.raises(ValueError, match=device):
        attention_call(b, cache=fake_cache(b, device))
    k = Fake((3, 2, 64), BF16)
    with pytest.raises(ValueError, match=device):
        b.kv_append(fake_cache(b, device), k, k, Fake((3,), torch.int64))


@pytest.mark.parametrize("bad", ["k", "v", "slots"])
def test_append_refuses_tensors_of_another_device(b, bad):
    a = {n: Fake((3, 2, 64), BF16, "cuda:1" if n == bad else "cuda:0") for n in ("k", "v")}
    slots = Fake((3,), torch.int64, "cuda:1" if bad == "slots" else "cuda:0")
    with pytest.raises(ValueError, match="cuda"):
        b.kv_append(fake_cache(b), a["k"], a["v"], slots)


@pytest.mark.parametrize("bad", range(10))
def test_plan_refuses_tensors_of_another_device(b, bad):
    shapes = [(2,), (2,), (2, 5), (7,), (1,)]
    dev = ["cuda:1" if i == bad else "cuda:0" for i in range(10)]
    a = [Fake(s, device=d) for s, d in zip(shapes, dev)]
    out = b.KvBatch(a[2], Fake((2,), device=dev[5]), Fake((3,), device=dev[6]), Fake((4,), torch.int64, dev[7]),
                    Fake((4,), device=dev[8]), Fake((2,), device=dev[9]), Fake((2,)))
    with pytest.raises(ValueError, match="cuda"):
        b.kv_plan(*a, tokens=4, page_size=16, out=out)


def test_cache_refuses_parts_that_do_not_belong_together(b):
    def cache(**change):
        c = b.empty_kv_cache(b.NVFP4, 4, 2, 64, page_size=16, device="cpu")
        for name, t in change.items():
            setattr(c.v, name, t)
        return c
    for change in (dict(scales=torch.empty((128, 4), dtype=torch.uint8, device="meta")),
                   dict(codes=torch.empty((128, 8), dtype=torch.int32, device="meta")),
                   dict(global_scale=torch.empty(1, device="meta")), dict(global_scale=torch.empty(1, dtype=torch.float64)),
                   dict(global_scale=torch.empty(2)), dict(scales=torch.empty((64, 4), dtype=torch.uint8))):
        c = cache(**change)
        with pytest.raises(ValueError):
            b.KvCache(c.k, c.v, kv_heads=2, page_size=16)
        with pytest.raises(ValueError):  # and of a cache whose parts were exchanged
            c.desc()
    assert cache(global_scale=torch.empty(1)).desc()


def attend(b, max_pages=2, scale=1.0):
    """bsfp_kv_attention over two requests at addresses that are never dereferenced."""
    from block_scaled_bit_fp_amd.kv import KvCacheDesc
    at = 0x10000
    k, v = (b.QTensorDesc(b.MXFP4, 4, 32, 4 * 2 * 16, 64, at, at, None, None, None) for _ in range(2))
    c = KvCacheDesc(C.pointer(k), C.pointer(v), 4, 2, 16)
    return b.lib().bsfp_kv_attention(at, 256, 3, 4, C.byref(c), at, max_pages, at, at, 2, 1, scale, 0, at, None, at,
                                     1 << 40, None)


@pytest.mark.parametrize("scale", [2.4e38, 3e38])
def test_attention_refuses_a_scale_that_overflows_in_log2_units(b, scale):
    assert attend(b, scale=scale) == ARG
    assert "scale" in b.lib().bsfp_last_error().decode()


def test_attention_refuses_tables_whose_keys_pass_31_bits(b):
    """Key numbers are 32-bit and run a few tiles past the last one."""
    for max_pages in ((1 << 27) - 511, 1 << 27, (1 << 31) - 1):
        assert attend(b, max_pages=max_pages) == UNSUPPORTED
        assert "keys" in b.lib().bsfp_last_error().decode()
