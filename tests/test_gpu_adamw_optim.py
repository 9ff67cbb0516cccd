"""The torch.optim front end of AdamW: training loops as a user writes them,
against the plain forms fed the same gradients."""
import numpy as np
import pytest

import adamw_common as A
from test_gpu_adamw import assert_state, dev, host

pytestmark = pytest.mark.gpu

F = np.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make_model(dtype):
    import torch
    torch.manual_seed(0)
    return torch.nn.Sequential(torch.nn.Linear(33, 129), torch.nn.LayerNorm(129), torch.nn.GELU(),
                               torch.nn.Linear(129, 7)).to("cuda", dtype)


def split(model):
    return [{"params": [p for p in model.parameters() if p.dim() > 1], "weight_decay": 0.1},
            {"params": [p for p in model.parameters() if p.dim() <= 1], "weight_decay": 0.0}]


@pytest.mark.parametrize("kind", ["f32", "f32-8", "master", "stochastic-8"])
def test_training_loop_with_groups_schedule_and_clipping(kind):
    """Forward, backward over two accumulated passes, clipped step, schedule:
    after every step all state equals the plain form's on the same gradients,
    and a state_dict taken mid-run continues bit-identically."""
    import torch
    from communication_compressed_distributed_02_amd.optim import AdamWOptimizer
    dt = torch.float32 if kind.startswith("f32") else torch.bfloat16
    kw = dict(lr=1e-2, max_norm=0.5, seed=11, state_bits=8 if kind.endswith("8") else 32,
              master=kind == "master", stochastic=kind.startswith("stochastic"))
    model = make_model(dt)
    opt = AdamWOptimizer(split(model), **kw)
    sched = torch.optim.lr_scheduler.LambdaLR(opt, [lambda t: 1 / (1 + t), lambda t: 0.5])
    groups = [i for i, g in enumerate(opt.param_groups) for _ in g["params"]]
    ref = A.Reference([host(p).ravel() for p in opt.params], opt.core.offsets, kw["state_bits"],
                      "f32" if dt == torch.float32 else "bf16", kw["master"], kw["stochastic"],
                      groups, 11)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def passes(m):
        for _ in range(2):
            x = torch.randn(16, 33, device="cuda", generator=gen).to(dt)
            (m(x).float() ** 2).mean().backward()

    for t in range(6):
        opt.zero_grad()
        passes(model)
        grads = [host(p.grad).ravel() for p in opt.params]
        rates = [g["lr"] for g in opt.param_groups]
        assert abs(rates[0] - 1e-2 / (1 + t)) < 1e-9 and abs(rates[1] - 5e-3) < 1e-9
        version = opt.params[0]._version
        opt.step(grad_scale=0.5)
        assert opt.params[0]._version > version
        sched.step()
        ref.step(grads, rates, [0.1, 0.0], 0.5, 0.5)
        want = ref.norm(grads, 0.5)
        assert abs(float(opt.norm) - want) <= 2 * A.U * want
        assert_state_of(opt, ref, "%s step %d" % (kind, t))
        if t == 2:
            saved = opt.state_dict()
            weights = [p.detach().clone() for p in opt.params]
            kept, rates2 = [], []
        if t > 2:
            kept.append([p.grad.clone() for p in opt.params])
            rates2.append(rates)
    other = make_model(dt)
    opt2 = AdamWOptimizer(split(other), **kw)
    for p, w in zip(opt2.params, weights):
        p.data.copy_(w)
    opt2.load_state_dict(saved)
    for grads, rates in zip(kept, rates2):
        for p, g in zip(opt2.params, grads):
            p.grad = g
        for g, r in zip(opt2.param_groups, rates):
            g["lr"] = r
        opt2.step(grad_scale=0.5)
    torch.cuda.synchronize()
    assert opt2.steps == opt.steps == (6, 0)
    for p, q in zip(opt.params, opt2.params):
        assert torch.equal(p, q)


def assert_state_of(opt, ref, where):
    """assert_state over the core's flat view of the model's tensors."""
    core = opt.core
    keep = core.params
    core.params = tuple(p.detach().reshape(-1) for p in opt.params)
    try:
        assert_state(core, ref, where)
    finally:
        core.params = keep


def test_against_torch_adamw_in_float64():
    """Five steps on given gradients against torch's own AdamW in float64: per
    step the fp32 form is within 3u|x| + 10u|up| + ... of the formulas from the
    same state, and m and v carry 3u and 4u of their sums a step, which the
    averages forget; 5 steps of at most lr = 1e-2 each, so x is within
    5 * (3u * 1.5 + 40u * 1e-2) of it."""
    import torch
    from communication_compressed_distributed_02_amd.optim import AdamWOptimizer
    torch.manual_seed(2)
    x = torch.rand(3000, device="cuda") - 0.5
    p, q = torch.nn.Parameter(x.clone()), torch.nn.Parameter(x.double())
    lr, wd = float(F(1e-2)), float(F(0.1))
    a = AdamWOptimizer([p], lr=lr, weight_decay=wd)
    b = torch.optim.AdamW([q], lr=lr, weight_decay=wd, betas=(float(A.B1), float(A.B2)),
                          eps=float(A.EPS))
    for _ in range(5):
        g = torch.rand(3000, device="cuda") + 0.5  # of one sign: no cancellation in m
        p.grad, q.grad = g, g.double()
        a.step()
        b.step()
    assert float((p.detach().double() - q.detach()).abs().max()) <= 5 * (4.5 + 0.4) * A.U


def test_missing_new_and_strided_gradients():
    import torch
    from communication_compressed_distributed_02_amd.optim import AdamWOptimizer
    ps = [torch.nn.Parameter(dev(np.linspace(-1, 1, 60, dtype=F)).view(6, 10)) for _ in range(3)]
    opt = AdamWOptimizer(ps, lr=1e-2, weight_decay=0.0)
    ref = A.Reference([host(p).ravel() for p in ps], opt.core.offsets)
    r = np.random.RandomState(3)
    for t in range(4):
        gs = [r.randn(60).astype(F) for _ in ps]
        for i, (p, g) in enumerate(zip(ps, gs)):
            p.grad = None if i == t else dev(g).view(6, 10)  # new memory every step
        # a gradient with other strides
        ps[(t + 1) % 3].grad = dev(gs[(t + 1) % 3]).view(6, 10).t().contiguous().t()
        if t < 3:
            gs[t] = None
        opt.step()
        ref.step(gs, 1e-2, 0.0)
        assert_state_of(opt, ref, "step %d" % t)
    # parameters that moved are found where they are
    moved = [p.data.clone() for p in ps]
    for p, m in zip(ps, moved):
        p.data = m
        p.grad = dev(np.ones(60, F)).view(6, 10)
    opt.step()
    ref.step([np.ones(60, F)] * 3, 1e-2, 0.0)
    assert_state_of(opt, ref, "moved")


def test_captured_optimizer_step():
    """step() captured on fixed gradients with the rates on the device; the
    gradients' contents and the rates change between replays."""
    import torch
    from communication_compressed_distributed_02_amd.optim import AdamWOptimizer
    ps = [torch.nn.Parameter(dev(np.full(n, 0.5, F))) for n in (5000, 77)]
    gs = [dev(np.zeros(n, F)) for n in (5000, 77)]
    for p, g in zip(ps, gs):
        p.grad = g
    opt = AdamWOptimizer([{"params": [ps[0]]}, {"params": [ps[1]], "weight_decay": 0.0}],
                         weight_decay=0.1, max_norm=1.0, state_bits=8, skip_nonfinite=True)
    ref = A.Reference([host(p) for p in ps], opt.core.offsets, 8, groups=[0, 1])
    rates = torch.zeros(2, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # a stream of its own, apart from the library's
        opt.step(lr=rates)
    norm = opt.norm
    r = np.random.RandomState(4)
    for k in range(5):
        new = [r.randn(g.numel()).astype(F) for g in gs]
        if k == 3:
            new[1][5] = np.inf
        for g, n in zip(gs, new):
            g.copy_(torch.from_numpy(n))
        lr = [1e-2 / (k + 1), 1e-3]
        rates.copy_(torch.tensor(lr))
        graph.replay()
        torch.cuda.synchronize()
        if k == 3:
            assert not np.isfinite(float(norm))
        else:
            ref.step(new, lr, [0.1, 0.0], 1.0)
            assert abs(float(norm) - ref.norm(new)) <= 2 * A.U * ref.norm(new)
        assert_state_of(opt, ref, "replay %d" % k)
    assert opt.steps == (4, 1)


def test_refusals():
    import torch
    from communication_compressed_distributed_02_amd.optim import AdamWOptimizer
    p = torch.nn.Parameter(torch.zeros(8, device="cuda"))
    opt = AdamWOptimizer([p])
    with pytest.raises(ValueError):
        opt.add_param_group({"params": [torch.nn.Parameter(torch.zeros(8, device="cuda"))]})
    with pytest.raises(ValueError):
        AdamWOptimizer([{"params": [p], "betas": (0.5, 0.9)}])
    with pytest.raises(ValueError):
        AdamWOptimizer([torch.nn.Parameter(torch.zeros(8))])
    with pytest.raises(ValueError):
        AdamWOptimizer([torch.nn.Parameter(torch.zeros(8, 8, device="cuda").t()[:4])])
    with pytest.raises(ValueError):
        AdamWOptimizer([])
    e = torch.nn.Embedding(5, 2, sparse=True, device="cuda")
    sparse = AdamWOptimizer(e.parameters())
    e(torch.tensor([1], device="cuda")).sum().backward()
    with pytest.raises(ValueError):
        sparse.step()
    with pytest.raises(ValueError):
        opt.load_state_dict(sparse.state_dict())
