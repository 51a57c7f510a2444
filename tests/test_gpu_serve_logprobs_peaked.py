"""token_logprobs (include/wbserve.h) of rows whose probability is one token's: log probabilities are at most 0, entropies at
least 0, and both within the bound of tests/test_gpu_serve_logprobs.py."""
import pytest

from tests.test_gpu_serve_logprobs import TYPES, run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,V,K", [(2000, 700, 8), (300, 5001, 0), (2, 140000, 20), (100, 128, 64)])
def test_signs(dtype, N, V, K):
    g = torch.Generator().manual_seed(V)
    x = torch.randn((N, V), generator=g)
    at = torch.randint(0, V, (N,), generator=g)
    x[torch.arange(N), at] += 20 + 20 * torch.rand(N, generator=g)
    x = x.to(TYPES[dtype]).cuda()
    lp, en, ids, tops = run(x, at.tolist(), K, rows=range(min(N, 60)))
    assert (lp <= 0).all() and (en >= 0).all() and (not K or (tops <= 0).all())
    lp, en, ids, tops = run(x, at.tolist(), K, scale=1e9, rows=range(min(N, 5)))
    assert (lp <= 0).all() and (en >= 0).all() and (not K or (tops <= 0).all())
