"""bench.py on several GPUs runs no kernel with TMA multicast: every rank has
chosen the forward without it before the first step is set up."""
import types

import pytest
import torch
import torch.distributed as dist

import bench
from long_context_sequence_seq_gb300 import build as B
from long_context_sequence_seq_gb300 import ulysses as U


class SetUp(Exception):
    pass


@pytest.mark.parametrize("world,want", [(1, []), (2, [2]), (8, [2])])
def test_ranks_choose_before_the_first_step(monkeypatch, world, want):
    chosen = []

    def step(*a, **k):
        raise SetUp

    monkeypatch.setenv("WORLD_SIZE", str(world))
    monkeypatch.setenv("RANK", str(world - 1))
    monkeypatch.setenv("LOCAL_RANK", str(world - 1))
    monkeypatch.setattr(dist, "init_process_group", lambda *a, **k: None)
    monkeypatch.setattr(torch.cuda, "set_device", lambda d: None)
    monkeypatch.setattr(U, "lib", lambda: None)
    monkeypatch.setattr(U, "set_kernel", chosen.append)
    monkeypatch.setattr(bench, "LayerStep", step)
    args = types.SimpleNamespace(workload="qwen3_4b_64k", seq_len=0, warmup=3, steps=1)
    with pytest.raises(SetUp):
        bench.gpu_arm(args)
    assert chosen == want and U.KERNEL_NO_MULTICAST == 2


def test_choices_the_library_takes():
    B.build()
    L = U.lib()
    try:
        for which in (U.KERNEL_NO_MULTICAST, U.KERNEL_SIMT, U.KERNEL_AUTO):
            assert L.ulysses_set_kernel(which) == U.OK
        for which in (-1, 3):
            assert L.ulysses_set_kernel(which) == U.ERR_INVALID
    finally:
        L.ulysses_set_kernel(U.KERNEL_AUTO)
