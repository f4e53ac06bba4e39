"""Where the outputs of the paged calls and of the rotation come from."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from bwd_tile_mean_gb300 import vsa
from tests.paged_ref import D, Pool
from tests.test_gpu_paged import BF

pytestmark = pytest.mark.gpu


def test_deterministic_fill_of_rows_left_unwritten():
    """torch.use_deterministic_algorithms fills uninitialised memory with NaN:
    the rows of q_out that no token has."""
    pool = Pool("bshd", BF, 4, 2, 16, 4, 2, [20], seed=1)
    cache = pool.cache()
    x = torch.ones(30, 4, D, dtype=BF, device="cuda")
    torch.full_like(x, 7.0)  # freed: what the allocator hands out next
    was = torch.are_deterministic_algorithms_enabled(), torch.utils.deterministic.fill_uninitialized_memory
    try:
        torch.use_deterministic_algorithms(True)
        torch.utils.deterministic.fill_uninitialized_memory = True
        q = cache.append(x[:, :2], x[:, :2], x, cu_seqlens=torch.tensor([0, 20], dtype=torch.int32, device="cuda"))
    finally:
        torch.use_deterministic_algorithms(was[0])
        torch.utils.deterministic.fill_uninitialized_memory = was[1]
    assert torch.isnan(q[20:]).all() and torch.equal(q[:20], x[:20])


def test_dispatch_modes_see_the_outputs():
    seen = []

    class Mode(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            seen.append(str(func))
            return func(*args, **(kwargs or {}))

    pool = Pool("bshd", BF, 4, 2, 16, 4, 2, [20], seed=1)
    cache, q = pool.cache(), torch.ones(1, 4, D, dtype=BF, device="cuda")
    with Mode():
        cache.attend(q)
    assert sum("empty" in f for f in seen) == 2, seen


def test_the_profiler_sees_the_outputs():
    rope, x = vsa.AxialRope((128,)), torch.ones(1, 3, 2, D, dtype=BF, device="cuda")
    at = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as p:
        rope.forward(x, positions=at)
    assert any("aten::empty" in e.key for e in p.key_averages())


def test_inference_tensors():
    pool = Pool("bshd", BF, 4, 2, 16, 4, 2, [20], seed=1)
    cache, q = pool.cache(), torch.ones(1, 4, D, dtype=BF, device="cuda")
    with torch.inference_mode():
        out = cache.attend(q)[0]
    assert out.is_inference() and not cache.attend(q)[0].is_inference()
