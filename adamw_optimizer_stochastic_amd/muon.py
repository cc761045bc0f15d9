"""MuonSR: a torch.optim.Optimizer over the fused Muon step.

Takes the arguments of torch.optim.Muon, for the 2-D parameters of hidden
layers (embeddings, the output layer, norms and biases belong to AdamWSR), and
this library's rounding: bf16 parameters are updated without an f32 master
copy, by stochastic rounding under key (seed, step) at each element's
position. Positions run over all parameters of the optimizer as in AdamWSR;
``base_offset`` moves them, so that the two optimizers of one model need not
share positions (give MuonSR the number of elements AdamWSR has).

For each matrix: m = momentum*m + g (f32), u = g + momentum*m (nesterov) or m,
p = p*(1 - lr*weight_decay) - lr*factor*O(u), O the Newton-Schulz
orthogonalisation. torch.optim.Muon keeps the average (1 - momentum)*m instead
and divides by max(|u|, eps) where this divides by |u| + eps: with a momentum
that stays the same the steps are the same but for eps, with one that changes
they are not (there the average's weight of old gradients stays, here their
sum's). All matrices of a group go through the products together,
which is what fills the chip with small ones. A step captured into a graph
repeats its number, learning rate and bits on every replay.
"""

import math
import operator

import torch

from . import ops
from .optim import _step_count

__all__ = ["MuonSR"]


def _checked(group):
    """A group's options as a step takes them, or an error."""
    o = {k: group[k] for k in ("lr", "weight_decay", "momentum", "nesterov", "ns_coefficients",
                               "eps", "ns_steps", "adjust_lr_fn", "rounding")}
    if isinstance(o["lr"], torch.Tensor):
        raise NotImplementedError("MuonSR: tensor lr is not supported")
    if not 0.0 <= o["lr"] < math.inf:
        raise ValueError(f"Invalid learning rate: {o['lr']}")
    if not 0.0 <= o["weight_decay"] < math.inf:
        raise ValueError(f"Invalid weight_decay value: {o['weight_decay']}")
    if not 0.0 <= o["momentum"] < 1.0:
        raise ValueError(f"Invalid momentum value: {o['momentum']}")
    if not 0.0 <= o["eps"] < math.inf:
        raise ValueError(f"Invalid epsilon value: {o['eps']}")
    if not 1 <= o["ns_steps"] <= 64:
        raise ValueError("ns_steps must be in [1, 64]")
    if o["rounding"] not in ("sr", "rn"):
        raise ValueError("rounding must be 'sr' or 'rn'")
    o["ns_steps"] = operator.index(o["ns_steps"])
    o["ns_coefficients"] = ops._coefficients(o["ns_coefficients"])
    if o["adjust_lr_fn"] is None:
        o["adjust_lr_fn"] = "original"
    ops.muon_lr_factor(1, 1, o["adjust_lr_fn"])
    return o


def _check_param(p):
    if p.dim() != 2:
        raise ValueError(f"MuonSR takes 2-D parameters (got shape {tuple(p.shape)})")
    if p.is_sparse or p.is_complex() or p.dtype not in (torch.float32, torch.bfloat16):
        raise NotImplementedError(f"MuonSR supports dense float32/bfloat16 params (got {p.dtype})")
    if max(p.shape) > ops.MUON_MAX_SIDE:
        raise ValueError(f"MuonSR takes sides of at most 2**20 (got shape {tuple(p.shape)})")


class MuonSR(torch.optim.Optimizer):
    def __init__(self, params, lr=1e-3, weight_decay=0.1, momentum=0.95, nesterov=True,
                 ns_coefficients=ops.NS_COEFFICIENTS, eps=1e-7, ns_steps=5, adjust_lr_fn=None,
                 *, seed=0, rounding="sr", base_offset=0):
        if not (isinstance(seed, int) and 0 <= seed < (1 << 32)):
            raise ValueError("seed must be an integer in [0, 2**32)")
        self.seed = seed
        self._base_index = {}
        self._next_index = ops._u64("base_offset", base_offset)
        defaults = _checked(dict(lr=lr, weight_decay=weight_decay, momentum=momentum,
                                 nesterov=nesterov, ns_coefficients=ns_coefficients, eps=eps,
                                 ns_steps=ns_steps, adjust_lr_fn=adjust_lr_fn, rounding=rounding))
        super().__init__(params, defaults)

    def add_param_group(self, param_group):
        super().add_param_group(param_group)
        group = self.param_groups[-1]
        try:   # (torch's own form of the group is what is checked; a refused one leaves again)
            group.update(_checked(group))
            for p in group["params"]:
                _check_param(p)
        except Exception:
            self.param_groups.pop()
            raise
        for p in group["params"]:
            self._base_index[p] = self._next_index
            self._next_index += p.numel()

    def base_index(self, p):
        """Global position of element 0 of parameter p."""
        return self._base_index[p]

    def _init_state(self, p):
        if len(self.state[p]) == 0:
            if p.is_cuda and torch.cuda.is_current_stream_capturing():
                raise RuntimeError("MuonSR: take one step before capturing one (a replay would "
                                   "start from a momentum of zeros every time)")
            self.state[p] = {"step": torch.tensor(0, dtype=torch.int64),
                             "momentum_buffer": torch.zeros(p.shape, dtype=torch.float32,
                                                            device=p.device)}

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        live = [[p for p in g["params"] if p.grad is not None] for g in self.param_groups]
        for p in (p for ps in live for p in ps):   # all of them, before the first moves
            if p.grad.is_sparse:
                raise NotImplementedError("MuonSR does not support sparse gradients")
            if not p.is_contiguous() or not p.grad.is_contiguous():
                raise NotImplementedError("MuonSR needs contiguous params and grads")
            self._init_state(p)
        for group, params in zip(self.param_groups, live):
            batches = {}   # (device, step) -> params
            for p in params:
                t = int(self.state[p]["step"]) + 1
                batches.setdefault((p.device, t), []).append(p)
            for (_, t), ps in batches.items():
                ops.muon_step(ps, [p.grad for p in ps],
                              [self.state[p]["momentum_buffer"] for p in ps],
                              [self._base_index[p] for p in ps], lr=group["lr"],
                              momentum=group["momentum"], nesterov=group["nesterov"],
                              weight_decay=group["weight_decay"], ns_steps=group["ns_steps"],
                              ns_coefficients=group["ns_coefficients"], eps=group["eps"],
                              adjust_lr=group["adjust_lr_fn"], step=t, seed=self.seed,
                              rounding=group["rounding"])
                for p in ps:
                    self.state[p]["step"].fill_(t)
        return loss

    def state_dict(self):
        sd = super().state_dict()
        sd["muon_sr"] = {"seed": self.seed}
        return sd

    def load_state_dict(self, state_dict):
        """Like torch's, except that the momentum stays float32 whatever the
        parameter dtype (torch's loader would cast it).

        Also takes a state of torch.optim.Muon, whose buffer is 1 - momentum times
        this one's and which counts no steps (here from 0); options it does not have
        stay as they are. A state that does not fit is refused before anything changes.
        """
        extra = state_dict.get("muon_sr")
        saved_state, saved_groups = state_dict.get("state", {}), state_dict["param_groups"]
        groups, loaded = [], []
        for group, saved in zip(self.param_groups, saved_groups):
            merged = {k: v for k, v in group.items() if k not in ("params", "param_names")} | saved
            groups.append(merged | _checked(merged))
            for p, pid in zip(group["params"], saved["params"]):
                st = saved_state.get(pid)
                if st is None:
                    continue
                m = st.get("momentum_buffer")
                if not isinstance(m, torch.Tensor) or m.numel() != p.numel():
                    raise ValueError("MuonSR: the state of a parameter of shape "
                                     f"{tuple(p.shape)} has no momentum_buffer of its size")
                ours = "step" in st
                loaded.append((p, _step_count(st["step"]) if ours else 0, m.detach().reshape(p.shape),
                               1.0 if ours else 1.0 - merged["momentum"]))
        if len(groups) == len(saved_groups):
            saved_groups = groups   # (a different number of groups is torch's to refuse)
        super().load_state_dict({**{k: v for k, v in state_dict.items() if k != "muon_sr"},
                                 "state": {}, "param_groups": saved_groups})
        for group in self.param_groups:
            for p in group["params"]:
                self.state.pop(p, None)
        for p, step, m, scale in loaded:
            self._init_state(p)
            self.state[p]["step"].fill_(step)
            self.state[p]["momentum_buffer"].copy_(m)
            if scale != 1.0:
                self.state[p]["momentum_buffer"].div_(scale)
        if extra is not None:
            self.seed = int(extra["seed"])
