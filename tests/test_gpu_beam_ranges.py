"""Selection at the ends of its arguments' ranges: temperatures and norms near fp32's largest value with
logits that differ by nats at them, and logits whose difference passes fp32."""
import math

import pytest
import torch

from tests import beam_ref as ref

pytestmark = pytest.mark.gpu

sd = pytest.importorskip("speculative_decoding_verification_logits_gb300")

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _check(dev, x, scores, k, T=1.0, norm=None, **more):
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    beams = sd.beam_select(x.to(dev), scores.to(dev), k, temperature=T, status=st,
                           norm=None if norm is None else norm.to(dev), **more)
    want = ref.select(x, scores, k, T=T, norm=norm, **more)
    ref.check_select(beams, want, k, norm)
    assert int(st) == want[2] == 0


def _wide(shape, dtype, seed):
    """Logits spread over the whole of fp32's range, each beam's over a part of its own."""
    g = torch.Generator().manual_seed(seed)
    x = (2 * torch.rand(shape, generator=g, dtype=torch.float64) - 1) * 3.3e38
    x *= 0.2 + 0.8 * torch.rand((*shape[:2], 1), generator=g, dtype=torch.float64)
    x[:, 0, 0], x[:, 0, -1] = 3.38e38, -3.38e38
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,W,V,k", [(2, 4, 700, 12), (1, 6, 40001, 24), (170, 3, 900, 9)])
@pytest.mark.parametrize("T", [1.0, 1e30, 1.3e36, 1.4e36, 2e37, 8.4e37, 1e38, 3.4e38])
def test_logits_over_the_whole_range(dev, dtype, B, W, V, k, T):
    x = _wide((B, W, V), dtype, V)
    g = torch.Generator().manual_seed(B)
    s = -4 * torch.rand((B, W), generator=g)
    _check(dev, x, s, k, T)
    _check(dev, x[:, :, 1:], s * 1e8, k, T, eos=3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,n", [(1e38, 1.0), (1.0, 1e38), (1e20, 2e18), (3e38, 1e-3), (1e-3, 3e38),
                                 (1e38, 1e-38), (1.2e-38, 1e38), (1.0, 1.7e38), (1e19, 8e18)])
def test_temperatures_and_norms_whose_quotients_leave_fp32(dev, dtype, T, n):
    # beams of one scale, and beside them one of an ordinary norm
    B, W, V, k = 2, 5, 1200, 17
    g = torch.Generator().manual_seed(int(math.log2(T) + 200))
    x = torch.randn((B, W, V), generator=g).double()
    x = (x * min(T * max(n, 1.0), 3e37) * 0.9).to(dtype)
    s = -4 * torch.rand((B, W), generator=g) * min(max(n, 1.0), 1e37)
    norm = n * (1 - 0.5 * torch.rand((B, W), generator=g))
    _check(dev, x, s, k, T, norm)
    norm[1, 2] = 1.0
    _check(dev, x, s, k, T, norm)


@pytest.mark.parametrize("T", [2e34, 1e35, 1e36])
def test_differences_that_pass_fp32_between_worse_beams(dev, T):
    # a beam's second token is 6e38 / T below its first, and still above all of another beam's
    V, k = 2000, 8
    x = torch.full((1, 3, V), -math.inf)
    x[0, 0, 7], x[0, 0, 1900] = 3.2e38, -3.2e38
    x[0, 1, ::8] = torch.randn(V // 8, generator=torch.Generator().manual_seed(1))
    s = torch.tensor([[0.0, -6.4e38 / T * 1.5, -math.inf]])
    b = sd.beam_select(x.to(dev), s.to(dev), k, temperature=T)
    assert b.parents[0].tolist() == [0, 0] + [1] * (k - 2) and b.tokens[0, :2].tolist() == [7, 1900]
    _check(dev, x, s, k, T)


@pytest.mark.parametrize("V", [1, 3, 5000])
def test_scores_over_norms_that_are_equal_tie_in_their_order(dev, V):
    # -n over n for n up to 256: finished beams, and beams that are sure of their token
    g = torch.Generator().manual_seed(V)
    B, W = 40, 32
    n = torch.stack([torch.randperm(256, generator=g)[:W] + 1 for _ in range(B)]).float()
    x = torch.full((B, W, V), -2e3)
    x[:, :, V // 2] = 0.0
    fin = (torch.rand((B, W), generator=g) < 0.5).to(torch.uint8)
    for unit in (1.0, 0.375, 3.0):
        s = -unit * n
        b = sd.beam_select(x.to(dev), s.to(dev), W, norm=n.to(dev), finished=fin.to(dev), eos=V - 1)
        assert b.parents.tolist() == [list(range(W))] * B
        assert torch.equal(b.scores.cpu(), s) and torch.equal(b.finished.cpu() > 0, (fin > 0) |
                                                              (b.tokens.cpu() == V - 1))
        _check(dev, x, s, W, norm=n, eos=0)
