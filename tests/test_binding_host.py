"""Host-side checks of the binding's descriptors (no GPU needed)."""
import torch

import block_scaled_bit_fp_amd as b


def test_a_tensor_without_codes_or_scales_has_null_pointers():
    """They reach the library, which answers with a status and a message."""
    codes, scales = torch.empty((4, 8), dtype=torch.int32), torch.empty((4, 2), dtype=torch.uint8)
    for c, s in ((None, scales), (codes, None), (None, None)):
        d = b.QuantizedTensor(b.MXFP4, 4, 64, c, s).desc()
        assert d.codes == (None if c is None else c.data_ptr()) and d.scales == (None if s is None else s.data_ptr())
