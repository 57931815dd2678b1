"""Refusals and build rules of the receiver's decode calls at their edges: host only, nothing here
launches a kernel."""
import pytest
import torch

from tests.test_decode_host import BAD, NOGPU, attn, call_attn, needs_no_gpu

LOWEST = float(torch.finfo(torch.float32).min)


@needs_no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(scale=3e38), BAD), (dict(scale=-3e38), BAD), (dict(scale=2e38), NOGPU),
    (dict(band_bias=3e38, band_width=1), BAD), (dict(band_bias=-LOWEST, band_width=9), BAD),
    (dict(band_bias=3e38, band_width=0), NOGPU), (dict(band_bias=2.3e38, band_width=9), NOGPU),
    (dict(band_bias=LOWEST, band_width=9), NOGPU), (dict(band_bias=LOWEST, band_width=0), NOGPU),
])
def test_scales_and_biases_at_the_types_limits(lib, kw, status):
    assert call_attn(lib, a=attn(**kw)) == status and lib.mf_last_error().decode()
