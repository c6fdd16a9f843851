"""The data-parallel step's clipping is a GPU kernel: asking for it on CPU tensors is refused when the step is built,
not at its first use, and without it nothing changes.  Its place in the step, after the all-reduce and the averaging,
is tested on two gloo ranks with a plain clipping in the kernel's place."""
import datetime
import os
import socket

import numpy as np
import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

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


class _PlainClip:
    """What lbq.GradClip does to one flat buffer, in fp64."""

    def __init__(self, flat):
        self.flat = flat

    def clip(self, max_norm, stream=None):
        norm = self.flat.double().norm()
        self.flat.mul_(torch.clamp(max_norm / (norm + 1e-6), max=1.0).float())
        return norm.float()


def _rank_grads(rank):
    """A rank's gradients: the ranks' differ in size and direction and partly cancel, so that neither rank's own norm,
    nor the norm of the sum where the mean is asked for, gives the right coefficient."""
    g = torch.Generator().manual_seed(5)
    a, b = torch.randn(4, 128, generator=g), torch.randn(64, 4, generator=g)
    g.manual_seed(6 + rank)
    return (1 - 3 * rank) * a + torch.randn(4, 128, generator=g), (2 + rank) * b + torch.randn(64, 4, generator=g)


def _worker(rank, world, port, average, max_norm, out_dir):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port), RANK=str(rank), WORLD_SIZE=str(world))
    dist.init_process_group("gloo", rank=rank, world_size=world, timeout=datetime.timedelta(seconds=60))
    try:
        step = DataParallelQLoRA(_layers(), average=average, grad_fn=lambda L, X, dY: (X, dY) + _rank_grads(rank),
                                 device="cpu")
        step.max_grad_norm, step._clip = max_norm, _PlainClip(step.flat)
        step.step([(torch.zeros(2, 128), torch.zeros(2, 64))])
        np.save(os.path.join(out_dir, f"flat_{rank}.npy"), step.flat.numpy())
        np.save(os.path.join(out_dir, f"norm_{rank}.npy"), step.grad_norm.numpy())
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("max_norm", [5.0, 1e6])
def test_two_ranks_clip_what_they_reduced(tmp_path, average, max_norm):
    """norm and coefficient are those of the reduced (and averaged) buffer, and both ranks end with the same bits."""
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    mp.start_processes(_worker, args=(2, port, average, max_norm, str(tmp_path)), nprocs=2, start_method="spawn",
                       join=True)
    flats = [np.load(tmp_path / f"flat_{r}.npy") for r in range(2)]
    norms = [np.load(tmp_path / f"norm_{r}.npy") for r in range(2)]
    assert np.array_equal(flats[0], flats[1]) and norms[0] == norms[1], "ranks disagree"
    total = sum(torch.cat([t.reshape(-1) for t in _rank_grads(r)]).double() for r in range(2))
    if average:
        total = total / 2
    norm = total.norm().item()
    # the sum of two fp32 values is rounded once (2^-24), halving is exact, so is the plain norm but for its rounding;
    # the product adds the coefficient's and its own rounding
    assert abs(float(norms[0]) - norm) <= 2 * 2.0 ** -24 * norm
    want = total.numpy() * min(1.0, max_norm / (norm + 1e-6))
    assert np.all(np.abs(flats[0] - want) <= 4 * 2.0 ** -24 * np.abs(want) + 1e-30)
    assert (norm > max_norm) == (max_norm == 5.0), "the case clips, or does not"
