"""Edges of the output-head losses' arguments on the host."""

import pytest

import test_head_host as host


@host.host_only
@pytest.mark.parametrize("tau", [1e-30, 1e-20, 1.0e-19, 1.9e19, 1e20, 3e38])
def test_temperatures_whose_square_is_no_normal_number(tau):
    # the losses are T^2 times a sum: inf or 0 times it, whatever they are
    for f in (host._kd_fwd, host._kd_bwd):
        assert f(tau=tau) == host.E_ARG, tau
