"""torch.optim front ends of the library's optimizers.

OneBitAdamOptimizer: 1-bit Adam over a list of ragged parameter tensors, n
simulated workers (below).  AdamWOptimizer: AdamW over parameters where they
lie, with states in 32 bits or in 8 (its own docstring).

1-bit Adam over a list of ragged parameter tensors, n simulated workers.

The parameters are moved once into the library's flat fp32 parameter buffer
and rebound as views of it, and every worker gets one flat gradient buffer
whose per-parameter views can be bound as the parameters' .grad (autograd
then accumulates into them in place).  A step therefore copies nothing: it
is one library call over the flat buffers.  The first `warmup_steps` steps
are full-precision Adam ("1-bit Adam ..." Abstract: warm-up phase), the rest
compression-phase steps with the variance frozen; the learning rate may
follow a schedule (the LIT-278 record notes that the frozen variance meets
learning-rate annealing in the compression phase).

Layout: every tensor starts at a multiple of 64 elements and is followed by
zero padding up to the next multiple of 64; the flat length is padded to a
multiple of 64 * n_workers.  Padding elements keep zero gradients.

It is a torch.optim.Optimizer with one parameter group: the learning rate is
read from param_groups[0]["lr"] at every step, so torch's LR schedulers
drive it, and state_dict() / load_state_dict() carry the library's whole
state (workspace bytes and step counters), so a run resumes bit-identically.
"""
import torch

from . import ob_adam as ob
from . import ob_adamw as oa


def flat_layout(numels, n_workers):
    """Start offset of every tensor and the padded flat length."""
    offsets = []
    off = 0
    for k in numels:
        offsets.append(off)
        off += -(-k // 64) * 64
    unit = 64 * n_workers
    d = max(unit, -(-off // unit) * unit)
    return offsets, d


class OneBitAdamOptimizer(torch.optim.Optimizer):
    def __init__(self, params, n_workers, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
                 warmup_steps=1, grad_dtype=torch.float32, lr_schedule=None):
        params = list(params)
        if not params:
            raise ValueError("no parameters")
        super().__init__(params, dict(lr=lr, betas=tuple(betas), eps=eps))
        if len(self.param_groups) != 1:
            raise ValueError("one parameter group")
        self.params = self.param_groups[0]["params"]
        dev = self.params[0].device
        for p in self.params:
            if p.dtype != torch.float32 or p.device != dev:
                raise ValueError("parameters must be float32 tensors on one device")
        if grad_dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("gradients are float32 or bfloat16")
        if warmup_steps < 1:
            raise ValueError("the variance is frozen after at least one warm-up step")
        self.n = n_workers
        self.lr_schedule = lr_schedule
        self.warmup_steps = warmup_steps
        self.grad_dtype = grad_dtype
        self.numels = [p.numel() for p in self.params]
        self.offsets, self.d = flat_layout(self.numels, n_workers)
        self._gt = ob.OB_GRAD_BF16 if grad_dtype == torch.bfloat16 else ob.OB_GRAD_F32
        self.core = ob.OneBitAdam(self.d, n_workers, self._gt, betas[0], betas[1], eps,
                                  device=dev)
        x = self.core.params_view()
        with torch.no_grad():
            for p, off, k in zip(self.params, self.offsets, self.numels):
                x[off:off + k].copy_(p.detach().reshape(-1))
        self._bind_params()
        self.grads = torch.zeros((n_workers, self.d), dtype=grad_dtype, device=dev)
        self.t = 0

    def _bind_params(self):
        x = self.core.params_view()
        for p, off, k in zip(self.params, self.offsets, self.numels):
            p.data = x[off:off + k].view(p.shape)

    def worker_grads(self, w):
        """Views of worker w's gradient buffer, one per parameter (its shape)."""
        g = self.grads[w]
        return [g[off:off + k].view(p.shape)
                for p, off, k in zip(self.params, self.offsets, self.numels)]

    def bind_worker(self, w):
        """Make worker w's views the parameters' .grad, so that a backward pass
        accumulates straight into worker w's buffer (float32 gradients only)."""
        if self.grad_dtype != torch.float32:
            raise ValueError("binding .grad needs float32 gradients; write bf16 ones into "
                             "worker_grads(w)")
        for p, gv in zip(self.params, self.worker_grads(w)):
            p.grad = gv

    def zero_grad(self, set_to_none=False):
        """Zero every worker's gradient buffer (the bound .grad views stay)."""
        self.grads.zero_()

    def current_lr(self):
        if self.lr_schedule is not None:
            return float(self.lr_schedule(self.t))
        return float(self.param_groups[0]["lr"])

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        lr = self.current_lr()
        bufs = list(self.grads.unbind(0))
        if self.t < self.warmup_steps:
            self.core.warmup_step(bufs, lr)
        else:
            self.core.compressed_step(bufs, lr)
        self.t += 1
        return loss

    @property
    def compressing(self):
        return self.t >= self.warmup_steps

    def flat_params(self):
        return self.core.params_view()

    def state_dict(self):
        """The library's state (workspace bytes on the CPU, counters) and the
        optimizer's own step count and learning rate."""
        data, counters = self.core.checkpoint("cpu")
        return {"workspace": data, "counters": counters, "t": self.t,
                "lr": self.param_groups[0]["lr"], "d": self.d, "n": self.n}

    def load_state_dict(self, state):
        if state["d"] != self.d or state["n"] != self.n:
            raise ValueError("state of a different layout (d=%d, n=%d)" % (state["d"], state["n"]))
        g = self.param_groups[0]
        self.core = ob.OneBitAdam(self.d, self.n, self._gt, g["betas"][0], g["betas"][1],
                                  g["eps"], device=self.params[0].device,
                                  checkpoint=(state["workspace"], tuple(state["counters"])))
        self._bind_params()
        self.t = state["t"]
        g["lr"] = state["lr"]


class AdamWOptimizer(torch.optim.Optimizer):
    """AdamW over parameters that stay where they are: contiguous float32 or
    bfloat16 tensors of one type on one GPU, their .grad of `grad_dtype`
    (default the same type).

    Groups (at most 32) may differ in lr and weight_decay, which are read from
    param_groups at every step, so torch's LR schedulers drive it; betas and eps
    are common.  state_bits, master, stochastic and seed as for ob_adamw.AdamW:
    with master, weights loaded into the model later are overwritten by the
    copies at the next step.  max_norm: clip
    by the global gradient norm (0: no clipping), without a host wait; the last
    norm is in `norm` on the device.  skip_nonfinite: a step whose gradients are
    not all finite changes nothing.  A parameter without a gradient is left as it
    is.  state_dict() / load_state_dict() carry the library's whole state and what it
    was made with, all of which but grad_dtype has to be the same where it is loaded."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2,
                 state_bits=32, master=False, stochastic=False, grad_dtype=None, max_norm=0.0,
                 skip_nonfinite=False, seed=0, stream=None):
        self._core = None
        super().__init__(params, dict(lr=lr, weight_decay=weight_decay))
        self.params = [p for g in self.param_groups for p in g["params"]]
        groups = [i for i, g in enumerate(self.param_groups) for _ in g["params"]]
        self.max_norm, self.skip_nonfinite, self.norm = max_norm, skip_nonfinite, None
        self._core = oa.AdamW([p.detach() for p in self.params], groups, len(self.param_groups),
                              grad_dtype, state_bits, master, stochastic, betas, eps, seed,
                              stream=stream)

    @property
    def core(self):
        """The ob_adamw.AdamW behind it."""
        return self._core

    def add_param_group(self, param_group):
        if self._core is not None:
            raise ValueError("the parameters are fixed when the optimizer is made")
        for k in param_group:
            if k not in ("params", "lr", "weight_decay"):
                raise ValueError("a group has its own lr and weight_decay only, not " + k)
        super().add_param_group(param_group)

    def grads(self):
        """The parameters' gradients as the library takes them."""
        out = []
        for p in self.params:
            g = p.grad
            if g is not None:
                if g.is_sparse:
                    raise ValueError("sparse gradients are not supported")
                if not g.is_contiguous():
                    g = g.contiguous()
            out.append(g)
        return out

    @torch.no_grad()
    def step(self, closure=None, grad_scale=1.0, lr=None, sumsq=None):
        """One step.  grad_scale: multiplies the gradients (1 / loss scale, 1 /
        accumulated passes).  lr: one rate per group in place of the groups' own, for
        a captured step a float32 device tensor.  sumsq: the squared norm to clip
        and skip by (a sum over ranks) as a float64 device scalar."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        if lr is None:
            lr = [float(g["lr"]) for g in self.param_groups]
        grads = self.grads()
        # the parameters as they lie now
        batch = self._core.bind(grads, self.params)
        self.norm = self._core.step(batch, lr, [g["weight_decay"] for g in self.param_groups],
                                    self.max_norm, grad_scale, self.skip_nonfinite, sumsq)
        torch.autograd.graph.increment_version(
            [p for p, g in zip(self.params, grads) if g is not None])
        return loss

    @property
    def steps(self):
        """(steps taken, steps skipped); waits for the GPU."""
        return self._core.steps

    def _config(self):
        """What the state depends on, in plain types: the powers of the betas are
        part of it, and the rest decides what its bytes mean and how it goes on."""
        core = self._core
        return {"state_bits": core.cfg.state_bits, "param_dtype": str(core.param_dtype),
                "master": bool(core.cfg.master), "stochastic": bool(core.cfg.stochastic),
                "betas": [core.cfg.beta1, core.cfg.beta2], "eps": core.cfg.eps,
                "seed": core.cfg.seed, "groups": list(core.groups)}

    def state_dict(self):
        """The library's state (workspace bytes on the CPU), what it was made with
        and the groups' rates."""
        return {"workspace": self._core.checkpoint("cpu"), "numels": list(self._core.numels),
                "config": self._config(),
                "param_groups": [{k: v for k, v in g.items() if k != "params"}
                                 for g in self.param_groups]}

    def load_state_dict(self, state):
        """A state_dict() of an optimizer made with the same arguments over
        parameters of the same sizes.  The state is loaded where it lies, so steps
        captured before go on from it."""
        if (state["numels"] != list(self._core.numels)
                or len(state["param_groups"]) != len(self.param_groups)):
            raise ValueError("state of other parameters")
        # a state saved before it had one is taken by its sizes
        for name, own in self._config().items():
            saved = state.get("config", {}).get(name, own)
            if saved != own:
                raise ValueError("state of an optimizer with %s %r, this one has %r"
                                 % (name, saved, own))
        self._core.load(state["workspace"])
        for g, saved in zip(self.param_groups, state["param_groups"]):
            g.update(saved)
