"""The binding of the cache and attention calls without a GPU: each call refuses host tensors, and a stream of
another device than the tensors'."""
from types import SimpleNamespace

import pytest
import torch

import hadamard_bit_quant_hbl_b200 as hbl


@pytest.mark.parametrize("call", [
    lambda s, c, i: hbl.hbl_kv_append(s, s, i, c, 16), lambda s, c, i: hbl.hbl_kv_gather(c, i, 2, 64, 16),
    lambda s, c, i: hbl.hbl_attn_decode(s, c, i[:, None], i, 2, 16), lambda s, c, i: hbl.hbl_attn_prompt(s, s, s, i, i)])
def test_host_tensors_are_refused(call):
    with pytest.raises(ValueError, match="CUDA tensor"):
        call(torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(1 << 16, dtype=torch.uint8),
             torch.zeros(4, dtype=torch.int32))


def test_a_stream_of_another_device_is_refused():
    # it would be made current on its own device, and the call would run on whatever stream the tensors' has
    hbl._load_torch()
    with pytest.raises(ValueError, match="stream of the tensors' device"):
        hbl._on(SimpleNamespace(device_index=1), 0)
