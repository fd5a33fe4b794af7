"""Which gradients expert_ffn_backward takes buffers for (no GPU): the binding's checks, before any library call."""
import pytest

torch = pytest.importorskip("torch")

from mixture_experts_ffn_12_b200 import api, build  # noqa: E402

BF16 = torch.bfloat16
E, R, D, F = 2, 6, 32, 48


def _z(*s, dtype=BF16):
    return torch.zeros(s, dtype=dtype)


@pytest.mark.parametrize("grads,match", [
    # CPU tensors: a call whose buffers are right gets as far as the device check
    ((None, None, None, None, None, None), "CUDA"),
    ((None, None, _z(E, D, F), None, None, _z(E, D)), "CUDA"),
    ((_z(E, F, D), None, None, None, None, None), "CUDA"),
    ((None, _z(E, D, F), None, None, None, None), "grads.w_up: shape"),
    ((None, None, None, None, _z(E, F), None), "grads.b_up is given without grads.w_up"),
    ((_z(E, F, D), None, None, _z(E, D), None, None), "grads.b_gate: shape"),
    ((None, None, _z(E, D, F, dtype=torch.float32), None, None, None), "grads.w_down: dtype"),
])
def test_gradient_buffers(grads, match):
    build.build()
    cfg = api.make_config(D, F, E, 2)
    w = api.ExpertWeights(_z(E, F, D), _z(E, F, D), _z(E, D, F), None, None, None)
    with pytest.raises(ValueError, match=match):
        api.expert_ffn_backward(cfg, _z(R, D), torch.zeros(E + 1, dtype=torch.int32), w, _z(R, 2, F), _z(R, F), _z(R, D),
                                grads=api.ExpertGrads(*grads))
