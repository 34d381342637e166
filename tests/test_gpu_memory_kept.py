"""What a norm, a rule and a cache were made of stays theirs when the caller's tensors are given other memory."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from expert_cache_host_layer_gb300.norm import RMSNorm
    from expert_cache_host_layer_gb300.paged_kv import KVBatch, KVPages
    from expert_cache_host_layer_gb300.router import Router

DEV = "cuda:0"


def others(t, n=16):
    """Tensors of t's size, one of which would get memory that was let go."""
    return [torch.full_like(t, 100) for _ in range(n)]


def test_a_norms_weight():
    weight = torch.nn.Parameter(torch.full((4096,), 3.0, device=DEV))
    norm, x = RMSNorm(4096, weight), torch.ones(2, 4096, device=DEV)
    out = torch.empty_like(x)
    weight.data = torch.full((4096,), 7.0, device=DEV)
    held = others(weight.data)
    norm.apply(x, out)
    assert torch.allclose(out, torch.full_like(out, 3.0), rtol=1e-5) and len(held) == 16
    norm.weight.fill_(2.0)  # in place
    norm.apply(x, out)
    assert torch.allclose(out, torch.full_like(out, 2.0), rtol=1e-5)


def test_a_weight_written_in_place():
    weight = torch.nn.Parameter(torch.full((64,), 3.0, device=DEV))
    norm, x = RMSNorm(64, weight), torch.ones(2, 64, device=DEV)
    with torch.no_grad():
        weight.fill_(5.0)
    norm.apply(x, x)
    assert torch.allclose(x, torch.full_like(x, 5.0), rtol=1e-5)


def test_a_rules_bias():
    bias = torch.zeros(1024, device=DEV)
    bias[[7, 500]] = 10.0
    router = Router(1024, 2, score="sigmoid", bias=bias)
    idx, w = torch.empty(3, 2, dtype=torch.int32, device=DEV), torch.empty(3, 2, device=DEV)
    bias.data = torch.arange(1024, device=DEV).float()
    held = others(bias)
    router.route(torch.zeros(3, 1024, device=DEV), idx, w)
    assert idx.tolist() == [[7, 500]] * 3 and len(held) == 16
    assert np.allclose(w.cpu().numpy(), 0.5)


def test_a_caches_pages():
    k, v = (torch.zeros(4, 1, 64, 64, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    pages = KVPages(k, v)
    k.data, v.data = (torch.zeros(1, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    held = others(pages.k)
    ints = [torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0, 5], [5], [[2]])]
    new = torch.randn(5, 1, 64, device=DEV).bfloat16()
    pages.append(KVBatch(*ints, 5, 5), new, -new)
    pages.check()
    assert torch.equal(pages.k[2, :, :5], new.transpose(0, 1)) and torch.equal(pages.v[2, :, :5], -new.transpose(0, 1))
    assert all((t == 100).all() for t in held)
