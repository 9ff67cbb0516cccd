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


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_go_on_from_a_loaded_state(oa, bits):
    """load_state_dict between replays of a captured step and eager ones: all of
    them continue from the loaded state, which takes no memory of its own."""
    import torch
    from communication_compressed_distributed_02_amd.optim import AdamWOptimizer
    sizes = [5000, 77, 1 << 20]
    start, grads = make_inputs(sizes, 31, 1)
    ps = [torch.nn.Parameter(dev(a)) for a in start]
    gs = [dev(g) for g in grads[0]]
    for p, g in zip(ps, gs):
        p.grad = g
    opt = AdamWOptimizer(ps, weight_decay=0.1, max_norm=1.0, state_bits=bits, seed=3)
    bound = opt.core.bind(gs)
    rate = torch.full((1,), 1e-2, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(lr=rate)

    ref = A.Reference(start, opt.core.offsets, bits, seed=3)
    for k in range(2):
        graph.replay()
        ref.step(grads[0], 1e-2, 0.1, 1.0)
        assert_state(opt.core, ref, "replay %d" % k)
    saved, weights = opt.state_dict(), [p.detach().clone() for p in ps]
    for _ in range(3):
        graph.replay()
    opt.step(lr=rate)
    assert opt.steps == (6, 0)
    torch.cuda.synchronize()
    before, place = torch.cuda.memory_allocated(), opt.core.workspace.data_ptr()
    torch.cuda.reset_peak_memory_stats()
    for w, p in zip(weights, ps):
        p.data.copy_(w)
    opt.load_state_dict(saved)
    assert opt.steps == (2, 0) and opt.core.workspace.data_ptr() == place
    assert torch.cuda.max_memory_allocated() - before < opt.core.ws_bytes
    for k in range(3):
        if k == 1:
            opt.core.step(bound, rate, 0.1, 1.0)  # bound before the load
        else:
            graph.replay()
        ref.step(grads[0], 1e-2, 0.1, 1.0)
        assert_state(opt.core, ref, "after the load, %d" % k)
    assert opt.steps == (5, 0)
    with pytest.raises(ValueError):
        opt.core.load(saved["workspace"][1:])
    assert opt.steps == (5, 0)


def test_state_loaded_on_another_stream(oa):
    """A plan on its own stream: the load waits for a replay behind work on the
    caller's stream, and for the bytes that the caller is still making."""
    import torch
    side, mine = torch.cuda.Stream(), torch.cuda.Stream()
    x, g = dev(np.ones(5000, F)), dev(np.ones(5000, F))
    big = torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    opt = oa.AdamW([x], stream=side)
    opt.step([g], 1e-3)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        opt.step([g], 1e-3)
    torch.cuda.synchronize()
    saved = opt.checkpoint("cuda")
    for _ in range(3):
        with torch.cuda.stream(mine):
            for _ in range(20):
                big.add_(1.0)
            graph.replay()
            late = torch.zeros_like(saved)
            late.copy_(saved)
            opt.load(late)
            assert opt.steps == (1, 0)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert opt.steps == (2, 0) and opt.check_guards() == -1


def test_states_of_other_optimizers_are_refused(oa):
    """A state_dict of other betas, eps, seed, rounding, groups, state width or
    parameter type changes nothing where it is refused; one of another gradient
    type, and one from before the configuration was saved, are taken."""
    import torch
    from communication_compressed_distributed_02_amd.optim import AdamWOptimizer

    def make(dtype=torch.bfloat16, split=1, **kw):
        ps = [torch.nn.Parameter(torch.ones(n, device="cuda", dtype=dtype)) for n in (300, 40)]
        for p in ps:
            p.grad_dtype = kw.get("grad_dtype", dtype)
            p.grad = torch.ones_like(p, dtype=p.grad_dtype)
        groups = [{"params": ps[:split]}, {"params": ps[split:]}]
        return AdamWOptimizer(groups, **kw)

    opt = make()
    opt.step()
    before = opt.core.checkpoint()
    for kw in ({"betas": (0.9, 0.99)}, {"betas": (0.8, 0.999)}, {"eps": 1e-6}, {"seed": 1},
               {"stochastic": True}, {"master": True}, {"state_bits": 8}, {"split": 0},
               {"dtype": torch.float32}):
        other = make(**kw)
        other.step()
        with pytest.raises(ValueError):
            opt.load_state_dict(other.state_dict())
        assert torch.equal(opt.core.checkpoint(), before), kw
    with pytest.raises(ValueError):
        opt.core.load(before.float())
    with pytest.raises(ValueError):
        oa.AdamW(opt.core.params, groups=[0, 1], checkpoint=before.float())
    other = make(grad_dtype=torch.float32)
    for _ in range(2):
        other.step()
    opt.load_state_dict(other.state_dict())
    assert opt.steps == (2, 0)
    old = {k: v for k, v in other.state_dict().items() if k != "config"}
    other.step()
    other.load_state_dict(old)
    assert other.steps == (2, 0)


def test_checkpoint_is_taken_before_later_calls_from_other_streams(oa):
    """A device copy asked for behind a few milliseconds of work on one stream,
    then a step from another: the copy is of the state before that step."""
    import torch
    side, mine = torch.cuda.Stream(), torch.cuda.Stream()
    x, g = dev(np.ones(5000, F)), dev(np.ones(5000, F))
    big = torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    opt = oa.AdamW([x], stream=side)
    for k in range(3):
        opt.step([g], 1e-3)
        before = host(opt.get("m", 0))
        with torch.cuda.stream(mine):
            for _ in range(20):
                big.add_(1.0)
            saved = opt.checkpoint("cuda")
        opt.step([g], 1e-3)
        after = host(opt.get("m", 0))
        with torch.cuda.stream(mine):
            saved = saved.cpu()
        again = oa.AdamW([x], stream=side, checkpoint=saved)
        assert again.steps == (2 * k + 1, 0) and opt.steps == (2 * k + 2, 0)
        assert A.same(host(again.get("m", 0)), before) and not A.same(after, before)


def test_calls_that_wait_are_refused_under_capture(oa):
    """Plans made, loaded, copied and asked for their counts while the current
    stream is captured, with the plan on that stream or on one of its own: each
    is refused, and the capture goes on with what it had."""
    import torch
    for own in (False, True):
        side, mine = torch.cuda.Stream(), torch.cuda.Stream()
        stream = side if own else mine
        x, g, y = (dev(np.ones(5000, F)) for _ in range(3))
        torch.cuda.synchronize()
        opt = oa.AdamW([x], stream=stream)
        saved = opt.checkpoint()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=mine):
            y.add_(1.0)
            for call in (opt.checkpoint, lambda: opt.checkpoint("cuda"), lambda: opt.load(saved),
                         lambda: opt.steps, opt.check_guards,
                         lambda: oa.AdamW([x], stream=stream), lambda: oa.GradNorm([x]),
                         lambda: oa.AdamW([x], stream=stream, checkpoint=saved)):
                with pytest.raises(RuntimeError):
                    call()
            opt.step([g], 1e-3)
        torch.cuda.synchronize()
        for k in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert float(y[0]) == 2.0 + k and opt.steps == (k + 1, 0)
