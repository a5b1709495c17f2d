"""The attention forward without TMA multicast gives the same bits as with it."""
import pytest
import torch

from long_context_sequence_seq_gb300 import ulysses as U
from tests.gpu_util import seq_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S,Hq,Hkv,D", [(1000, 8, 2, 128), (517, 4, 2, 64), (384, 6, 2, 128)])
@pytest.mark.parametrize("fused", [False, True])
def test_same_results_without_multicast(S, Hq, Hkv, D, fused):
    q, k, v, _ = seq_inputs(S, Hq, Hkv, D, "bf16")
    cu = torch.tensor([0, S // 3, S], dtype=torch.int32, device="cuda")
    run = lambda: (U.layer_fwd_fused if fused else U.layer_fwd)(q, k, v, 1, Hq, cu_seqlens=cu)  # noqa: E731
    n0 = U.launch_count()
    auto = run()
    launches = U.launch_count() - n0
    U.set_kernel(U.KERNEL_NO_MULTICAST)
    try:
        alone = run()
        U.check()
    finally:
        U.set_kernel(U.KERNEL_AUTO)
    assert U.launch_count() - n0 == 2 * launches
    assert torch.equal(auto[0], alone[0]) and torch.equal(auto[1], alone[1])
    assert bool(torch.isfinite(alone[0]).all())
