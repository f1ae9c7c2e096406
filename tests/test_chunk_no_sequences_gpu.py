"""The schedule of the chunk attention without sequences: its records are all zero, and neither array is read."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("parts", [1, 76, 1024])
def test_records_without_sequences(parts):
    import paged_mla_decode_10_gb300 as M
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.mla_check_device_error()
    for total in (0, 9):                       # 9: padding only
        for _ in range(20):
            # a schedule of other lengths leaves its sums in the shared memory that the next one finds
            cu = torch.tensor([0, 50, 300], dtype=torch.int32, device="cuda")
            M.mla_chunk_get_metadata(cu, torch.tensor([900, 4000], dtype=torch.int32, device="cuda"), 300, 16, 1)
            md = M.mla_chunk_get_metadata(one, one[:0], total, 16, 1, num_parts=parts)
            assert md.shape == (parts, 8) and not md.any()
    assert M.mla_check_device_error() == 0


def test_null_arrays_without_sequences():
    from paged_mla_decode_10_gb300 import _lib
    md = torch.full((76, 8), 7, dtype=torch.int32, device="cuda")
    rc = _lib.load().mla_chunk_get_metadata(None, None, 0, 0, 16, 1, 1, 76, ctypes.c_void_p(md.data_ptr()),
                                            ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0 and not md.any()
