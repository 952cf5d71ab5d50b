"""Where fp8_quantize_experts may write: experts that share memory are refused,
every layout whose experts lie apart passes that check."""
import pytest
import torch

import post_weight_quantization_16_amd as g

E4 = torch.float8_e4m3fn


def _out(E, N, K, strides):
    size = sum((n - 1) * s for n, s in zip((E, N, K), strides)) + 1
    flat = torch.zeros(size, dtype=torch.uint8)
    return g.Fp8Experts(torch.as_strided(flat, (E, N, K), strides).view(E4),
                        torch.ones(E, -(-N // 128), -(-K // 128)))


@pytest.mark.parametrize("E,N,K,strides", [(3, 4, 8, (0, 8, 1)), (3, 4, 8, (31, 8, 1)), (2, 4, 8, (16, 16, 1)), (3, 4, 8, (7, 64, 1)),
                                           (4, 1, 8, (0, 8, 1)), (2, 1, 8, (7, 99, 1)), (3, 4, 8, (60, 30, 1)), (9, 3, 8, (10, 80, 1))])
def test_experts_that_share_memory(E, N, K, strides):
    with pytest.raises(ValueError, match="overlap"):
        g.fp8_quantize_experts(torch.zeros(E, N, K), out=_out(E, N, K, strides))


@pytest.mark.parametrize("E,N,K,strides", [(3, 4, 8, (32, 8, 1)), (3, 4, 8, (8, 24, 1)), (3, 4, 8, (16, 48, 1)), (3, 4, 8, (100, 16, 1)),
                                           (1, 4, 8, (0, 8, 1)), (2, 1, 8, (8, 0, 1)), (2, 4, 8, (70, 20, 1)), (8, 3, 8, (10, 80, 1))])
def test_experts_that_lie_apart(E, N, K, strides):
    flat = [set(range(e * strides[0] + n * strides[1], e * strides[0] + n * strides[1] + K)) for e in range(E) for n in range(N)]
    assert len(set().union(*flat)) == E * N * K
    with pytest.raises(ValueError) as e:     # of the host: refused for that alone
        g.fp8_quantize_experts(torch.zeros(E, N, K), out=_out(E, N, K, strides))
    assert "overlap" not in str(e.value)
