"""The largest sizes that the decoder's entry points take, decided on the host."""
import pytest

from precision_transformer_gemms_gb300 import lpq
from test_decoder_abi import on_cpu, route, VALID


@pytest.mark.parametrize("m", [1 << 30, (1 << 30) - 3, 1 << 40])
def test_route_refuses_more_tokens_than_a_grid_has(m):
    """Two CTAs a token, in clusters of eight for four: a grid holds 2^31 - 1."""
    assert route(m=m) == lpq.ERR_SHAPE


@on_cpu
def test_route_takes_all_that_it_has():
    assert route(m=(1 << 30) - 4) in VALID
