"""Outputs over the weights that later rows still read are refused. No call reaches the device."""
import pytest

from tests import test_layer_abi as abi


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


def test_add_norm(ops):
    at = abi.at
    for kw in (dict(o=at(0)), dict(h=at(0)), dict(h=at(0) + 8176), dict(o=at(0) - 4 * 4096 + 16), dict(post_w=at(6), o=at(6) + 4096),
               dict(post_w=at(6), h=at(6)), dict(post_w=at(6), h=at(6), o=0)):
        abi.refused(ops, abi.add_norm(ops, **kw), "norm weight")
