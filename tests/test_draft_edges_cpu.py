"""Refusals of the distillation loss's temperature, on the CPU."""
import pytest

import test_draft_cpu as base
import vocab_argmax_amd as vpa


@pytest.mark.parametrize("t", [0.0, -1.0, 2.0 ** -101, 1e-45, float("inf"), float("nan")])
def test_temperatures_that_are_refused(t):
    for call in (base.distill, base.backward, base.at_once):
        assert call(t=t) == vpa.VPA_ERR_INVALID
        assert "temperature" in vpa.last_error()
