"""The attention binding's two ways (C++ and Python) on unusual arguments."""
import pytest
import torch

import implicit_gemm_nhwc_amd as igc
from implicit_gemm_nhwc_amd import attention as binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class NoTruth:
    def __bool__(self):
        raise ValueError("neither true nor false")


@pytest.mark.parametrize("way", ["C++", "Python"])
def test_arguments_without_a_truth_value(way, monkeypatch):
    """Their own exception is raised, and the next call is not disturbed."""
    assert binding._fast is not None
    if way == "Python":
        monkeypatch.setattr(binding, "_fast", None)
    q = torch.randn(1, 4, 2, 64, device=DEV).to(torch.bfloat16)
    table = igc.rope_table(4, 64, device=DEV)
    for call in (lambda: igc.cross_attention(q, q, q, return_lse=NoTruth()),
                 lambda: igc.qk_norm_rope(q, q_table=table, interleaved=NoTruth()),
                 lambda: igc.qk_norm_rope_bwd(q, None, q, q_table=table, interleaved=NoTruth())):
        with pytest.raises(ValueError, match="neither true nor false"):
            call()
        assert torch.isfinite(igc.cross_attention(q, q, q)).all()


@pytest.mark.parametrize("way", ["C++", "Python"])
def test_truth_values_of_any_type(way, monkeypatch):
    if way == "Python":
        monkeypatch.setattr(binding, "_fast", None)
    q = torch.randn(1, 4, 2, 64, device=DEV).to(torch.bfloat16)
    table = igc.rope_table(4, 64, device=DEV)
    assert isinstance(igc.cross_attention(q, q, q, return_lse=[]), torch.Tensor)
    assert len(igc.cross_attention(q, q, q, return_lse=[0])) == 2
    assert torch.equal(igc.qk_norm_rope(q, q_table=table, interleaved="yes"),
                       igc.qk_norm_rope(q, q_table=table, interleaved=True))
