"""CPU checks of the ft_kv calls and their torch wrapper beside tests/test_kv_abi.py."""
import pytest

ft = pytest.importorskip("expert_cache_host_layer_gb300")


def test_a_stream_that_does_not_capture_has_no_number():
    assert ft.ft_stream_capture(0) == 0
