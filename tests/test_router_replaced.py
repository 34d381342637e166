"""CPU check: a rule's bias is not let go before the cache's stream is past its last reader."""
import pytest

pytest.importorskip("torch")
pipeline = pytest.importorskip("expert_cache_host_layer_gb300.pipeline")


class Bias:
    def __init__(self, log):
        self.log = log

    def record_stream(self, stream):
        self.log.append(("recorded", stream))

    def dim(self):
        return 1


class Rule:
    num_experts, top_k, index, c = 8, 2, 0, "struct"

    def __init__(self, bias):
        self.bias = bias


def test_a_replaced_rules_bias_is_recorded_on_the_caches_stream(monkeypatch):
    log = []
    monkeypatch.setattr(pipeline, "ft_cache_set_router", lambda handle, router: log.append(("set", router)))
    cache = object.__new__(pipeline.ExpertCache)
    cache.E, cache.k, cache.L, cache.handle, cache.router, cache.stream = 8, 2, 3, 0, None, "compute"
    cache.pool = type("Pool", (), {"get_device": staticmethod(lambda: 0)})
    cache.set_router(Rule(Bias(log)))
    assert log == [("set", "struct")]
    cache.set_router(Rule(None))
    assert log[1:] == [("set", "struct"), ("recorded", "compute")]  # after the library has made the stream wait
    cache.set_router(None)
    assert log[3:] == [("set", None)]
