"""Arguments of the position bias beyond what the C entries hold, and calls without scores' batch."""
import pytest
import torch

import adaptive_gradient_summation_gb300 as ags

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("kw", [dict(offset=2 ** 64), dict(offset=2 ** 64 + 3), dict(offset=2 ** 63), dict(offset=-2 ** 63 - 1),
                                dict(max_distance=2 ** 64 + 128), dict(max_distance=-2 ** 64 + 128)])
def test_numbers_that_would_wrap_are_refused(native, kw):
    """2^64 is not offset 0, and 2^64 + 128 not distance 128."""
    table, x = torch.randn(32, 3, device=DEV), torch.randn(2, 3, 4, 8, device=DEV)
    for call in (lambda: ags.relative_position_bias(table, 4, 8, **kw), lambda: ags.relative_position_bias(table, 4, 8, scores=x, **kw),
                 lambda: ags.relative_position_bias_backward(x, 32, **kw)):
        with pytest.raises(ValueError, match="64 bits"):
            call()


def test_numbers_of_buckets_that_would_wrap_are_refused(native):
    d = torch.empty(2, 0, 4, 8, device=DEV)  # (no heads: nothing is allocated for them)
    for buckets in (2 ** 31, 2 ** 32 + 32):
        with pytest.raises(ValueError):
            ags.relative_position_bias_backward(d, buckets)


@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_an_empty_batch_writes_nothing(native, dtype):
    """It is no call for the bias alone, for which the output would hold a value of every head, query
    and key: the output's place is the middle of a buffer with room for them."""
    table = torch.randn(32, 3, device=DEV)
    room = torch.full((3 * 4 * 5 * 3,), 7.0, dtype=dtype, device=DEV)
    out = room[60:60].view(0, 3, 4, 5)
    scores = torch.empty(0, 3, 4, 5, dtype=dtype, device=DEV)
    assert ags.relative_position_bias(table, 4, 5, scores=scores, out=out) is out
    lib = ags.load_library()
    code = {FP32: 0, BF16: 1}[dtype]
    st = lib.adasum_relative_position_bias(table.data_ptr(), 32, 3, 0, 1, 128, 0, 4, 5, table.data_ptr(), 0, 60, 20, 5, code,
                                           room.data_ptr() + 60 * room.element_size(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert (room == 7).all()
    # the bias alone does write there
    alone = torch.full((3 * 4 * 5,), 7.0, device=DEV)
    st = lib.adasum_relative_position_bias(table.data_ptr(), 32, 3, 0, 1, 128, 0, 4, 5, None, 0, 0, 0, 0, 0, alone.data_ptr(),
                                           torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(alone.view(3, 4, 5), ags.relative_position_bias(table, 4, 5))
