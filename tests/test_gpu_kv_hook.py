"""bsfp_time_next_launch times qmv, qmm and qmm_dense: a call of the paged cache in between leaves the pair."""
import ctypes as C

import pytest
import torch

from test_gpu_kv import NVFP4, build, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_lens", [[1, 1], [40, 30]])
def test_a_pending_event_pair_outlasts_the_cache_calls(bsfp, q_lens):
    rt = C.CDLL("libamdhip64.so")
    rt.hipEventCreate.argtypes = [C.POINTER(C.c_void_p)]
    rt.hipEventElapsedTime.argtypes = [C.POINTER(C.c_float), C.c_void_p, C.c_void_p]
    rt.hipEventDestroy.argtypes = [C.c_void_p]
    ev = [C.c_void_p(), C.c_void_p()]
    for e in ev:
        assert rt.hipEventCreate(C.byref(e)) == 0
    cache, batch, q = build(bsfp, NVFP4, [100, 80], q_lens, 4, 2, 64, 16, seed=8)
    w = bsfp.quantize(rand((512, 1024), 1), NVFP4)
    x = rand((1, 1024), 2)
    ms = C.c_float()
    bsfp.time_next_launch(ev[0].value, ev[1].value)
    try:
        bsfp.kv_append(cache, rand((1, 2, 64), 3), rand((1, 2, 64), 4), torch.zeros(1, dtype=torch.int64, device="cuda"))
        bsfp.kv_attention(q, cache, batch)
        torch.cuda.synchronize()
        taken = rt.hipEventElapsedTime(C.byref(ms), ev[0], ev[1]) == 0
        rt.hipGetLastError()  # events that were never recorded are an error, which would come back later
        bsfp.qmv(x, w)
        torch.cuda.synchronize()
        assert not taken
        assert rt.hipEventElapsedTime(C.byref(ms), ev[0], ev[1]) == 0 and 0.0 < ms.value < 100.0
    finally:
        bsfp.time_next_launch(None, None)
        for e in ev:
            rt.hipEventDestroy(e)
