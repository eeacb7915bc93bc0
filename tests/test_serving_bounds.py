"""Refusals of the serving operators beyond test_serving_abi.py, on the CPU."""
import pytest

from lm_causal_depthwise_b200 import api, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load()


def test_debug_withhold_refuses(lib):
    assert lib.rglru_debug_withhold(-2) == api.ERR_INVALID_ARG
    assert lib.rglru_debug_withhold(-1) == api.OK
    with pytest.raises(api.RGLRUError):
        api.debug_withhold(-5)
