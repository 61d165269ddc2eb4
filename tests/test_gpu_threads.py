"""Decodes of two plans from two host threads at once."""

import numpy as np
import pytest

from tests.test_gpu_paged_edges import at_once

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tau", [0.0, 0.002])
def test_decodes_of_two_plans_in_two_threads(cuda_device, tau):
    # a short and a long cache: score slots, and so shared memory, differ
    import torch
    from loop_aware_quantized_b200 import LOOPKV_Q4, Plan
    from loop_aware_quantized_b200 import loopkv as lk
    dev, H, D = cuda_device, 2, 128
    g = torch.Generator(device=dev).manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    cells, made = np.zeros(1, np.int32), []
    for n in (64, 16384):
        plan = Plan(1, 1, H, D, np.array([n], np.int32), np.array([LOOPKV_Q4], np.uint8), tau=tau, device=dev)
        plan.append(cells, rand(1, 1, H, n, D), rand(1, 1, H, n, D))
        q = rand(1, 1, H, D)
        want, out, stream = plan.decode(cells, q), torch.zeros((1, 1, H, D), device=dev), torch.cuda.Stream(dev)
        args = (plan.handle, lk._np_ptr(cells), 1, 1, q.data_ptr(), out.data_ptr(), None, None, 0, None, stream.cuda_stream)
        made.append((plan, q, want, out, stream, args))
    torch.cuda.synchronize()
    found = at_once([lambda a=m[-1]: lk.loopkv_decode(*a) for m in made], 3000)
    torch.cuda.synchronize()
    assert found == [[], []]
    for plan, _, want, out, *_ in made:
        assert (out == want).all()
        plan.close()
