"""Decoder.step's checks of its inputs, without a GPU."""
from types import SimpleNamespace

import pytest
import torch

from head_sparse_paged_b200.runner import Decoder

BF = torch.bfloat16


def decoder():
    d = Decoder.__new__(Decoder)
    d.w = SimpleNamespace(num_seqs=3, num_q_heads=8, num_kv_heads=2, head_dim=64)
    d.device = torch.device("cpu")
    return d


def good():
    return {"q": torch.zeros(3, 8, 64, dtype=BF), "k_new": torch.zeros(3, 2, 64, dtype=BF),
            "v_new": torch.zeros(3, 2, 64, dtype=BF)}


def test_inputs_of_the_right_kind_pass():
    decoder().check_inputs(**good())
    decoder().check_inputs(**{**good(), "q": torch.zeros(8, 3, 64, dtype=BF).transpose(0, 1)})   # strides are copied


@pytest.mark.parametrize("name", ["q", "k_new", "v_new"])
def test_inputs_that_a_copy_would_cast_or_broadcast_are_refused(name):
    t = good()[name]
    for bad in (t.float(), t.half(), t[:1], t[0], t[:, :1], t[..., :1], t.reshape(-1), t.unsqueeze(0),
                torch.zeros(4, *t.shape[1:], dtype=BF), t.to("meta")):
        with pytest.raises(ValueError, match=name):
            decoder().check_inputs(**{**good(), name: bad})
