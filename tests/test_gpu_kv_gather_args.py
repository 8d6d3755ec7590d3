"""kq_kv_gather_q4 takes its number of rows from the places: what is no tensor of them is refused as such."""
import pytest

import quantized_weight_matmul_q4_gb300 as kq

pytestmark = pytest.mark.gpu


def test_places_that_are_no_tensor_of_places():
    import torch
    cache = torch.zeros(kq.kv_cache_q4_shape(2, 1, 16, 64), dtype=torch.uint8, device="cuda")
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    for bad in (None, [0, 1], torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64, device="cuda")):
        with pytest.raises(TypeError, match="positions"):
            kq.kq_kv_gather_q4(cache, table, bad)
    K, V = kq.kq_kv_gather_q4(cache, table, torch.tensor([3], dtype=torch.int32, device="cuda"))
    assert K.shape == V.shape == (1, 1, 64) and not K.any() and not V.any()
