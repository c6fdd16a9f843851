"""The data-parallel step's clipping is a GPU kernel: asking for it on CPU tensors is refused when the step is built,
not at its first use, and without it nothing changes."""
import pytest
import torch

from qlora_quantized_linear_b200.dp import AdapterLayer, DataParallelQLoRA


class _Weight:
    n, k = 64, 128


def _layers():
    return [AdapterLayer(_Weight(), torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(64, 4, dtype=torch.bfloat16), 2.0)]


def test_clipping_needs_a_gpu():
    with pytest.raises(ValueError, match="CUDA"):
        DataParallelQLoRA(_layers(), device="cpu", max_grad_norm=1.0)


def test_no_clipping_by_default():
    def grads(L, X, dY):
        return X, dY, torch.full((4, 128), 3.0), torch.full((64, 4), -2.0)

    step = DataParallelQLoRA(_layers(), grad_fn=grads, device="cpu")
    step.step([(torch.zeros(2, 128), torch.zeros(2, 64))])
    assert step.grad_norm is None
    assert bool((step.layers[0].dA == 3.0).all()) and bool((step.layers[0].dB == -2.0).all())
