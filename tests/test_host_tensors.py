"""Tensors that are not on a GPU are refused before anything is allocated for the call."""
import pytest
import torch

from gated_delta_rule_35_amd import binding

x = torch.zeros(1, 4, 1, 128, dtype=torch.bfloat16)
g = torch.zeros(1, 4, 1)
w = torch.ones(128)
CALLS = [
    lambda: binding.kda_gdr_fwd(x, x, x, g, g, 1.0, final_state=True),
    lambda: binding.kda_gdr_bwd(x, x, x, g, g, 1.0, x, d_initial_state=True),
    lambda: binding.kda_gdr_decode(x[0], x[0], x[0], g[0], g[0], 1.0, None),
    lambda: binding.kda_qk_norm(x, x),
    lambda: binding.kda_qk_norm_bwd(x, x, x, x, q_weight=w, k_weight=w),
]


@pytest.mark.parametrize("call", range(len(CALLS)))
def test_refused_before_anything_is_allocated(call, monkeypatch):
    def no(*a, **kw):
        raise AssertionError("allocated before the refusal")

    monkeypatch.setattr(binding, "_new", no)
    monkeypatch.setattr(binding, "_scratch", no)
    with pytest.raises(ValueError, match="on the GPU"):
        CALLS[call]()
