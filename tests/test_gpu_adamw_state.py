"""AdamW plans against what a program does around them: parameters and state
written as soon as a plan exists, state brought in and taken out between steps
and replays."""
import numpy as np
import pytest

import adamw_common as A
from test_gpu_adamw import assert_state, dev, host, make_inputs

pytestmark = pytest.mark.gpu

F = np.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(scope="module")
def oa():
    from communication_compressed_distributed_02_amd import ob_adamw
    return ob_adamw


def test_parameters_and_copies_may_be_written_once_the_plan_exists(oa):
    """Copies taken on a stream of the plan's own hold the parameters as they
    were, and what the caller writes next, on its own stream, stays."""
    import torch
    n = (1 << 27) + 777
    x = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    opt = oa.AdamW([x], master=True, stream=side)
    x.fill_(7.0)
    copies = opt.views()["master"][:n]
    assert bool((copies == 0.5).all())
    opt.close()
    del opt, copies
    x.fill_(0.5)
    torch.cuda.synchronize()
    opt = oa.AdamW([x], master=True, stream=side)
    copies = opt.views()["master"][:n]
    copies.fill_(3.0)
    torch.cuda.synchronize()
    assert bool((copies == 3.0).all())
