"""GB300 (sm_103a) fused offline-RL train step: HER relabel + IQL value update.

A thin Python binding over the C ABI of include/ofrl.h.  Every function
marshals torch CUDA tensors into device pointers and calls the library on
the current torch stream; all arithmetic runs in the library's CUDA kernels.
There is no CPU path: if libofrl.so is missing, importing the binding's
calls raises.

Functions (same names as the C entry points, without the ofrl_ prefix):
  Context(...)                  ofrl_create / ofrl_destroy / ofrl_poll_status
  her_relabel(...)              HER index sampling + gather + relabel
  iql_value_fwd_bwd(...)        V forward + expectile loss + V backward
  expectile_loss(...)           expectile loss and dL/dV
  adv_weighted_policy(...)      softmax(beta * clamp(Q - V, -10, 10)), argmax
  budgeted_clip_saxpy(...)      budgeted per-source clip + SAXPY, norms
  adam_step(...)                Adam with the safety clip
  train_step(...)               the fused step composed of the above
  DeltaRule(...)                ofrl_delta_create / _destroy / _poll_status
  delta_forward(...)            gated delta rule over packed episodes
  delta_backward(...)           its gradients
  delta_step(...)               one token for each environment
  CausalConv(...)               ofrl_conv_create / _destroy / _poll_status
  conv_forward(...)             short causal convolution over packed episodes
  conv_backward(...)            its gradients
  conv_step(...)                one token for each environment
  SelectiveScan(...)            ofrl_scan_create / _destroy / _poll_status
  scan_forward(...)             selective scan over packed episodes
  scan_backward(...)            its gradients
  scan_step(...)                one token for each environment
  BlockNorm(...)                ofrl_norm_create / _destroy
  gated_norm(...)               norm of a block's output with its gate
  gated_norm_backward(...)      its gradients
  residual_norm(...)            residual + scale x, and its norm
  residual_norm_backward(...)   its gradients
  TensorList(...)               ofrl_tensors_create / _destroy
  global_norm(...)              2-norm over many tensors
  global_norm_clip(...)         the norm, and every tensor clipped by it
"""
import ctypes as C
import struct
from dataclasses import dataclass, field
from typing import List, Optional, Sequence

import torch

from . import _abi
from ._abi import (HER_EPISODE, HER_FINAL, HER_FUTURE, HER_RANDOM, PREC_BF16, PREC_FP32,  # noqa: F401
                   STAT_BAD_ACTION, STAT_BAD_INDEX, STAT_NONFINITE_GRAD, STAT_SANITIZED, STAT_TIMEOUT, OfrlError)

STRATEGY = {"final": HER_FINAL, "future": HER_FUTURE, "random": HER_RANDOM, "episode": HER_EPISODE}
PRECISION = {"fp32": PREC_FP32, "bf16": PREC_BF16}
BUDGET = (0.70, 0.15, 0.10, 0.05)


def n_params(state_dim: int, hidden: int) -> int:
    return hidden * state_dim + hidden + hidden * hidden + hidden + hidden + 1


def _ptr(t: Optional[torch.Tensor], dtype=None, name="tensor", host_ok=False):
    """Address of a CUDA tensor; with host_ok also of a pinned CPU tensor (page-locked host memory the
    kernels read or write in place over the host link)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not (t.is_cuda or (host_ok and t.is_pinned())):
        raise TypeError(f"{name} must be a CUDA tensor" + (" or a pinned CPU tensor" if host_ok else ""))
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return C.c_void_p(t.data_ptr())


def _host_ptr(t: Optional[torch.Tensor], name="tensor"):
    """A page-locked float32 CPU tensor (the graph's host copies need pinned memory)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.is_cuda or not t.is_pinned():
        raise TypeError(f"{name} must be a pinned CPU tensor")
    if t.dtype != F32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 tensor")
    return C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


F32, I32, BF16 = torch.float32, torch.int32, torch.bfloat16


@dataclass
class Replay:
    """Replay buffer (device tensors): states/next_states [capacity, stride]."""
    states: torch.Tensor
    next_states: torch.Tensor
    actions: torch.Tensor
    rewards: torch.Tensor
    dones: torch.Tensor
    state_dim: int
    goal_dim: int
    episode_ends: Optional[torch.Tensor] = None

    def c(self):
        cap, stride = self.states.shape
        ne = 0 if self.episode_ends is None else int(self.episode_ends.numel())
        return _abi.Replay(_ptr(self.states, F32, "states"), _ptr(self.next_states, F32, "next_states"),
                           _ptr(self.actions, I32, "actions"), _ptr(self.rewards, F32, "rewards"),
                           _ptr(self.dones, F32, "dones"), _ptr(self.episode_ends, I32, "episode_ends"),
                           cap, ne, self.state_dim, stride, self.goal_dim)


@dataclass
class HerConfig:
    batch: int
    her_count: int
    strategy: str = "future"
    goal_threshold: float = 0.01
    seed: int = 0

    def c(self):
        return _abi.HerCfg(self.batch, self.her_count, STRATEGY[self.strategy], self.goal_threshold,
                           self.seed & ((1 << 64) - 1))


@dataclass
class Batch:
    """Relabelled batch (device tensors), written by her_relabel / train_step."""
    states: torch.Tensor
    next_states: torch.Tensor
    actions: torch.Tensor
    rewards: torch.Tensor
    dones: torch.Tensor
    src_idx: torch.Tensor
    donor_idx: torch.Tensor

    @classmethod
    def empty(cls, batch: int, stride: int, device="cuda"):
        f = dict(device=device, dtype=F32)
        i = dict(device=device, dtype=I32)
        return cls(torch.empty(batch, stride, **f), torch.empty(batch, stride, **f), torch.empty(batch, **i),
                   torch.empty(batch, **f), torch.empty(batch, **f), torch.empty(batch, **i),
                   torch.empty(batch, **i))

    def c(self):
        return _abi.Batch(_ptr(self.states, F32, "batch.states"), _ptr(self.next_states, F32, "batch.next_states"),
                          _ptr(self.actions, I32, "batch.actions"), _ptr(self.rewards, F32, "batch.rewards"),
                          _ptr(self.dones, F32, "batch.dones"), _ptr(self.src_idx, I32, "batch.src_idx"),
                          _ptr(self.donor_idx, I32, "batch.donor_idx"), self.states.shape[1])


@dataclass
class VNet:
    """One V network's trainable state: params, Adam moments m and v, step t; optionally a Polyak target copy
    that train_step moves toward the weights after every update (target = (1 - polyak) target + polyak params)."""
    params: torch.Tensor
    m: torch.Tensor
    v: torch.Tensor
    tau: float
    t: int = 0
    target: Optional[torch.Tensor] = None
    polyak: float = 0.0

    @classmethod
    def from_params(cls, params: torch.Tensor, tau: float, polyak: Optional[float] = None):
        p = params.detach().to(device="cuda", dtype=F32).contiguous().clone()
        tgt = p.clone() if polyak is not None else None
        return cls(p, torch.zeros_like(p), torch.zeros_like(p), float(tau), 0, tgt, float(polyak or 0.0))

    def c(self):
        return _abi.VNet(_ptr(self.params, F32, "params"), _ptr(self.m, F32, "m"), _ptr(self.v, F32, "v"),
                         self.t, self.tau, _ptr(self.target, F32, "target"), self.polyak)


@dataclass
class Opt:
    lr: float = 3e-4
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.0
    max_grad_norm: float = 1.0
    beta: float = 3.0
    budget: Sequence[float] = BUDGET
    alpha: Sequence[float] = (1.0, 1.0, 1.0, 1.0)
    weight_clamp_max_abs: float = 0.0    # > 0: |weight| bound after every Adam update
    sanitize_sources: bool = False       # non-finite gradient-source elements count as 0

    def c(self):
        b = (C.c_float * 4)(*[float(x) for x in (list(self.budget) + [0.0] * 4)[:4]])
        a = (C.c_float * 4)(*[float(x) for x in (list(self.alpha) + [0.0] * 4)[:4]])
        return _abi.Opt(self.lr, self.beta1, self.beta2, self.eps, self.weight_decay, self.max_grad_norm,
                        self.beta, b, a, self.weight_clamp_max_abs, 1 if self.sanitize_sources else 0)


# V forward/backward implementations (OFRL_VNET_* in ofrl.h)
VNET_PATHS = {"auto": 0, "tc_fused": 1, "tc_layered": 2, "cuda_cores": 3}


class Context:
    """Device workspace for one V-network shape (ofrl_create); the only allocation."""

    def __init__(self, state_dim: int, hidden: int, num_actions: int, prec: str = "fp32",
                 max_batch: int = 16384, max_nets: int = 1):
        self._lib = _abi.load()
        self.shape = _abi.VShape(state_dim, hidden, num_actions, PRECISION[prec])
        self.state_dim, self.hidden, self.num_actions, self.prec = state_dim, hidden, num_actions, prec
        self.max_batch, self.max_nets = max_batch, max_nets
        self.n_params = n_params(state_dim, hidden)
        h = C.c_void_p()
        _abi.check("ofrl_create", self._lib.ofrl_create(C.byref(self.shape), max_batch, max_nets, C.byref(h)))
        self.handle = h

    def close(self):
        if self.handle is not None and self.handle.value:
            _abi.check("ofrl_destroy", self._lib.ofrl_destroy(self.handle))
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def poll_status(self, stream=None):
        words = (C.c_int32 * _abi.STAT_WORDS)()
        _abi.check("ofrl_poll_status", self._lib.ofrl_poll_status(self.handle, _stream(stream), words))
        return {"nonfinite_grad": words[_abi.STAT_NONFINITE_GRAD], "bad_action": words[_abi.STAT_BAD_ACTION],
                "bad_index": words[_abi.STAT_BAD_INDEX], "timeout": words[_abi.STAT_TIMEOUT],
                "sanitized": words[_abi.STAT_SANITIZED]}

    def workspace_bytes(self) -> int:
        return int(self._lib.ofrl_workspace_bytes(C.byref(self.shape), self.max_batch, self.max_nets))

    def select_vnet_path(self, path: str):
        """Which V forward/backward implementation later calls take: auto, tc_fused, tc_layered, cuda_cores."""
        _abi.check("ofrl_select_vnet_path", self._lib.ofrl_select_vnet_path(self.handle, VNET_PATHS[path]))

    def vnet_path(self, n_nets: int = 1) -> str:
        """The implementation a train step of n_nets networks takes on this context."""
        k = int(self._lib.ofrl_vnet_path(self.handle, n_nets))
        names = {v: n for n, v in VNET_PATHS.items()}
        if k not in names:
            raise ValueError(f"ofrl_vnet_path: invalid arguments (n_nets={n_nets})")
        return names[k]


def her_relabel(ctx: Context, replay: Replay, her: HerConfig, step: int, out: Batch, stream=None):
    r, h, b = replay.c(), her.c(), out.c()
    _abi.check("ofrl_her_relabel", ctx._lib.ofrl_her_relabel(ctx.handle, C.byref(r), C.byref(h), step,
                                                              C.byref(b), _stream(stream)))


def her_relabel_sources(ctx: Context, replay: Replay, her: HerConfig, step: int, src_idx, out: Batch,
                        is_weights=None, is_weights_out=None, stream=None):
    """her_relabel with the caller's (e.g. PER-sampled) source of every row; HER rows get importance weight 1."""
    r, h, b = replay.c(), her.c(), out.c()
    _abi.check("ofrl_her_relabel_sources", ctx._lib.ofrl_her_relabel_sources(
        ctx.handle, C.byref(r), C.byref(h), step, _ptr(src_idx, I32, "src_idx"), _ptr(is_weights, F32, "is_weights"),
        C.byref(b), _ptr(is_weights_out, F32, "is_weights_out"), _stream(stream)))


def episode_ends_append(ctx: Context, dones, first_index: int, episode_ends, num_episodes, stream=None):
    """Append the exclusive end of every done transition among the n = dones.numel() new ones stored at
    first_index.. to episode_ends (device int32, in order), growing the device counter num_episodes."""
    _abi.check("ofrl_episode_ends_append", ctx._lib.ofrl_episode_ends_append(
        ctx.handle, _ptr(dones, F32, "dones"), int(first_index), int(dones.numel()), _ptr(episode_ends, I32, "episode_ends"),
        _ptr(num_episodes, I32, "num_episodes"), int(episode_ends.numel()), _stream(stream)))


def iql_value_fwd_bwd(ctx: Context, params, states, q_taken, tau: float, v_out, loss_out, grad_out,
                      stream=None):
    batch = int(q_taken.numel())
    _abi.check("ofrl_iql_value_fwd_bwd", ctx._lib.ofrl_iql_value_fwd_bwd(
        ctx.handle, _ptr(params, F32, "params"), _ptr(states, F32, "states"), states.shape[1], batch,
        _ptr(q_taken, F32, "q_taken"), tau, _ptr(v_out, F32, "v_out"), _ptr(loss_out, F32, "loss_out"),
        _ptr(grad_out, F32, "grad_out"), _stream(stream)))


def forward_values(ctx: Context, params, states, v_out, stream=None):
    """V(s) of every row of `states` [batch, stride] into v_out [batch] (forward only)."""
    _abi.check("ofrl_forward_values", ctx._lib.ofrl_forward_values(
        ctx.handle, _ptr(params, F32, "params"), _ptr(states, F32, "states"), states.shape[1],
        int(states.shape[0]), _ptr(v_out, F32, "v_out"), _stream(stream)))


def iql_target(ctx: Context, params, next_states, rewards, dones, gamma: float, target_out, v_next_out=None,
               stream=None):
    """target_out = rewards + gamma (1 - dones) V(next_states); V(s') into v_next_out when given."""
    _abi.check("ofrl_iql_target", ctx._lib.ofrl_iql_target(
        ctx.handle, _ptr(params, F32, "params"), _ptr(next_states, F32, "next_states"), next_states.shape[1],
        _ptr(rewards, F32, "rewards"), _ptr(dones, F32, "dones"), int(next_states.shape[0]), gamma,
        _ptr(v_next_out, F32, "v_next_out"), _ptr(target_out, F32, "target_out"), _stream(stream)))


def noalloc_max_batch(state_dim: int, hidden: int, num_actions: int, prec: str = "fp32") -> int:
    """Largest batch iql_value_fwd_bwd_noalloc accepts for this shape."""
    shape = _abi.VShape(state_dim, hidden, num_actions, PRECISION[prec])
    return int(_abi.load().ofrl_noalloc_max_batch(C.byref(shape)))


def iql_value_fwd_bwd_noalloc(state_dim: int, hidden: int, num_actions: int, params, states, q_taken,
                              tau: float, v_out, loss_out, grad_out, prec: str = "fp32", stream=None):
    """iql_value_fwd_bwd for callers that may not allocate device memory.

    No Context: the library's own fixed scratch array is used (see the C
    header), so nothing is allocated.  Calls that overlap on the GPU share
    that scratch and race: issue them on one stream.
    """
    lib = _abi.load()
    shape = _abi.VShape(state_dim, hidden, num_actions, PRECISION[prec])
    batch = int(q_taken.numel())
    _abi.check("ofrl_iql_value_fwd_bwd_noalloc", lib.ofrl_iql_value_fwd_bwd_noalloc(
        C.byref(shape), _ptr(params, F32, "params"), _ptr(states, F32, "states"), states.shape[1], batch,
        _ptr(q_taken, F32, "q_taken"), tau, _ptr(v_out, F32, "v_out"), _ptr(loss_out, F32, "loss_out"),
        _ptr(grad_out, F32, "grad_out"), _stream(stream)))


def expectile_loss(ctx: Context, q_taken, v, tau: float, loss_out, dv_out=None, stream=None):
    _abi.check("ofrl_expectile_loss", ctx._lib.ofrl_expectile_loss(
        ctx.handle, _ptr(q_taken, F32, "q_taken"), _ptr(v, F32, "v"), int(v.numel()), tau,
        _ptr(loss_out, F32, "loss_out"), _ptr(dv_out, F32, "dv_out"), _stream(stream)))


def adv_weighted_policy(ctx: Context, q, v, beta: float, pi_out, argmax_out=None, stream=None):
    b, a = q.shape
    _abi.check("ofrl_adv_weighted_policy", ctx._lib.ofrl_adv_weighted_policy(
        ctx.handle, _ptr(q, F32, "q"), _ptr(v, F32, "v"), b, a, beta, _ptr(pi_out, F32, "pi_out"),
        _ptr(argmax_out, I32, "argmax_out"), _stream(stream)))


def budgeted_clip_saxpy(ctx: Context, sources: List[torch.Tensor], budget_frac, alpha, max_grad_norm: float,
                        grad_out, norms_out=None, stream=None):
    k = len(sources)
    n = int(sources[0].numel())
    ptrs = (C.c_void_p * k)(*[_ptr(s, F32, "source").value for s in sources])
    bf = (C.c_float * k)(*[float(x) for x in budget_frac[:k]])
    al = (C.c_float * k)(*[float(x) for x in alpha[:k]])
    _abi.check("ofrl_budgeted_clip_saxpy", ctx._lib.ofrl_budgeted_clip_saxpy(
        ctx.handle, ptrs, bf, al, k, n, max_grad_norm, _ptr(grad_out, F32, "grad_out"),
        _ptr(norms_out, F32, "norms_out"), _stream(stream)))


def adam_step(ctx: Context, p, g, m, v, t: int, opt: Opt, grad_norm=None, stream=None):
    o = opt.c()
    _abi.check("ofrl_adam_step", ctx._lib.ofrl_adam_step(
        ctx.handle, _ptr(p, F32, "p"), _ptr(g, F32, "g"), _ptr(m, F32, "m"), _ptr(v, F32, "v"), int(p.numel()),
        t, C.byref(o), _ptr(grad_norm, F32, "grad_norm"), _stream(stream)))


def train_step(ctx: Context, replay: Replay, her: HerConfig, step: int, batch: Batch, q, nets: List[VNet],
               opt: Opt, aux: Optional[List[List[torch.Tensor]]] = None, v_out=None, pi_out=None,
               argmax_out=None, loss_out=None, norms_out=None, grad_out=None, stream=None):
    """One fused step; increments every net's t."""
    r, h, b, o = replay.c(), her.c(), batch.c(), opt.c()
    n_nets = len(nets)
    cn = (_abi.VNet * n_nets)(*[x.c() for x in nets])
    n_aux = 0 if not aux else len(aux[0])
    aux_arr = None
    if n_aux:
        flat = [_ptr(t, F32, "aux").value for per in aux for t in per]
        aux_arr = (C.c_void_p * len(flat))(*flat)
    _abi.check("ofrl_train_step", ctx._lib.ofrl_train_step(
        ctx.handle, C.byref(r), C.byref(h), step, C.byref(b), _ptr(q, F32, "q", host_ok=True), cn, n_nets, C.byref(o),
        aux_arr, n_aux, _ptr(v_out, F32, "v_out"), _ptr(pi_out, F32, "pi_out"),
        _ptr(argmax_out, I32, "argmax_out"), _ptr(loss_out, F32, "loss_out", host_ok=True),
        _ptr(norms_out, F32, "norms_out", host_ok=True), _ptr(grad_out, F32, "grad_out"), _stream(stream)))
    for k in range(n_nets):
        nets[k].t = cn[k].t


class StepPlan:
    """train_step with every argument marshalled once.

    Per call only the step index, the Q pointer and the optional auxiliary
    source pointers change; the networks' t counters live in the C array and
    advance there.  Same semantics as train_step.
    """

    def __init__(self, ctx: Context, replay: Replay, her: HerConfig, batch: Batch, nets: List[VNet], opt: Opt,
                 n_aux: int = 0, v_out=None, pi_out=None, argmax_out=None, loss_out=None, norms_out=None,
                 grad_out=None):
        self.ctx, self.nets = ctx, nets
        self._keep = (replay, batch, nets, v_out, pi_out, argmax_out, loss_out, norms_out, grad_out)
        self.r, self.h, self.b, self.o = replay.c(), her.c(), batch.c(), opt.c()
        self.n_nets = len(nets)
        self.cn = (_abi.VNet * self.n_nets)(*[x.c() for x in nets])
        self.n_aux = n_aux
        self.aux_arr = (C.c_void_p * max(1, self.n_nets * n_aux))()
        self.outs = [_ptr(v_out, F32), _ptr(pi_out, F32), _ptr(argmax_out, I32), _ptr(loss_out, F32, host_ok=True),
                     _ptr(norms_out, F32, host_ok=True), _ptr(grad_out, F32)]
        self.fn = ctx._lib.ofrl_train_step
        self.rp, self.hp, self.bp, self.op = C.byref(self.r), C.byref(self.h), C.byref(self.b), C.byref(self.o)

    def run(self, step: int, q: torch.Tensor, aux=None, stream=None):
        if self.n_aux:
            flat = [t.data_ptr() for per in aux for t in per]
            for i, p in enumerate(flat):
                self.aux_arr[i] = p
        code = self.fn(self.ctx.handle, self.rp, self.hp, step, self.bp, C.c_void_p(q.data_ptr()), self.cn,
                       self.n_nets, self.op, self.aux_arr if self.n_aux else None, self.n_aux, *self.outs,
                       _stream(stream))
        if code != _abi.OK:
            _abi.check("ofrl_train_step", code)

    def sync_t(self):
        for k in range(self.n_nets):
            self.nets[k].t = self.cn[k].t

    def reload_t(self):
        """Take each network's t from the VNet objects (after steps made by other means, e.g. a StepGraph)."""
        for k in range(self.n_nets):
            self.cn[k].t = self.nets[k].t

    def kernels(self) -> int:
        """Kernel launches one run() makes (4, or 3 when the reduce and Adam run as one launch)."""
        return int(self.ctx._lib.ofrl_train_step_kernels(self.ctx.handle, self.bp, self.h.batch, self.n_nets))


def target_ema(params, target, polyak: float, stream=None):
    """target = (1 - polyak) target + polyak params, element-wise (Polyak averaging of a target network)."""
    if params.numel() != target.numel():
        raise ValueError("params and target differ in size")
    _abi.check("ofrl_target_ema", _abi.load().ofrl_target_ema(
        _ptr(params, F32, "params"), _ptr(target, F32, "target"), int(params.numel()), polyak, _stream(stream)))


class StepGraph:
    """train_step captured once as a CUDA graph; launch() replays it as a given step.

    Same semantics as train_step: per launch the step index, and optionally the Q tensor and the auxiliary
    sources, change; each network's t advances.  Every other tensor is the one given here (keep them alive).
    One graph launch on the host per step.
    """

    def __init__(self, ctx: Context, replay: Replay, her: HerConfig, batch: Batch, nets: List[VNet], opt: Opt, q,
                 aux=None, v_out=None, pi_out=None, argmax_out=None, loss_out=None, norms_out=None, grad_out=None,
                 q_host=None, loss_host=None, norms_host=None):
        """q, loss_out and norms_out may be pinned CPU tensors, as for train_step (Q staged by the relabel,
        loss and norms written in place).  q_host / loss_host / norms_host (pinned CPU tensors, with device
        q, loss_out, norms_out): the graph also copies Q in from q_host and the loss and norms out to
        loss_host / norms_host; replay it with launch_io."""
        self.ctx, self.nets = ctx, nets
        self._keep = [replay, batch, nets, q, aux, v_out, pi_out, argmax_out, loss_out, norms_out, grad_out,
                      q_host, loss_host, norms_host]
        self.r, self.h, self.b, self.o = replay.c(), her.c(), batch.c(), opt.c()
        self.n_nets = len(nets)
        self.cn = (_abi.VNet * self.n_nets)(*[x.c() for x in nets])
        self.n_aux = 0 if not aux else len(aux[0])
        self.aux_arr = (C.c_void_p * max(1, self.n_nets * self.n_aux))()
        if self.n_aux:
            for i, t in enumerate(t for per in aux for t in per):
                self.aux_arr[i] = _ptr(t, F32, "aux").value
        handle = C.c_void_p()
        args = (ctx.handle, C.byref(self.r), C.byref(self.h), C.byref(self.b), _ptr(q, F32, "q", host_ok=True), self.cn,
                self.n_nets, C.byref(self.o), self.aux_arr if self.n_aux else None, self.n_aux,
                _ptr(v_out, F32, "v_out"), _ptr(pi_out, F32, "pi_out"), _ptr(argmax_out, I32, "argmax_out"),
                _ptr(loss_out, F32, "loss_out", host_ok=True), _ptr(norms_out, F32, "norms_out", host_ok=True),
                _ptr(grad_out, F32, "grad_out"))
        self.io = q_host is not None or loss_host is not None or norms_host is not None
        if self.io:
            _abi.check("ofrl_step_graph_create_io", ctx._lib.ofrl_step_graph_create_io(
                *args, _host_ptr(q_host, "q_host"), _host_ptr(loss_host, "loss_host"),
                _host_ptr(norms_host, "norms_host"), C.byref(handle)))
        else:
            _abi.check("ofrl_step_graph_create", ctx._lib.ofrl_step_graph_create(*args, C.byref(handle)))
        self.handle = handle
        self.fn = ctx._lib.ofrl_step_graph_launch
        self.fn_io = ctx._lib.ofrl_step_graph_launch_io

    def launch_io(self, step: int, q_host=None, aux=None, loss_host=None, norms_host=None, stream=None):
        """Replay as step `step` with this step's host buffers (pinned CPU tensors; None keeps the previous)."""
        arr = None
        if aux is not None:
            self._keep.append(aux)
            for i, t in enumerate(t for per in aux for t in per):
                self.aux_arr[i] = t.data_ptr()
            arr = self.aux_arr
        for t in (q_host, loss_host, norms_host):
            if t is not None:
                self._keep.append(t)
        code = self.fn_io(self.handle, step, _host_ptr(q_host, "q_host"), arr, _host_ptr(loss_host, "loss_host"),
                          _host_ptr(norms_host, "norms_host"), _stream(stream))
        if code != _abi.OK:
            _abi.check("ofrl_step_graph_launch_io", code)
        if len(self._keep) > 64:
            del self._keep[14:-8]

    def launch(self, step: int, q=None, aux=None, stream=None):
        arr = None
        if aux is not None:
            self._keep.append(aux)
            for i, t in enumerate(t for per in aux for t in per):
                self.aux_arr[i] = t.data_ptr()
            arr = self.aux_arr
        if q is not None:
            self._keep[3] = q
        code = self.fn(self.handle, step, C.c_void_p(q.data_ptr()) if q is not None else None, arr,
                       _stream(stream))
        if code != _abi.OK:
            _abi.check("ofrl_step_graph_launch", code)
        if len(self._keep) > 64:
            del self._keep[14:-8]

    def sync_t(self):
        for k in range(self.n_nets):
            self.nets[k].t = self.cn[k].t

    def close(self):
        if self.handle:
            self.ctx._lib.ofrl_step_graph_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- sequence memory (gated delta rule) --------------------------------------------------------------------------

DTYPE = {"fp32": _abi.DTYPE_F32, "bf16": _abi.DTYPE_BF16}
_TORCH_DTYPE = {"fp32": F32, "bf16": BF16}
_TENSOR = torch.Tensor      # looked up for every argument of every call


class DeltaRule:
    """Workspace of the gated delta rule for one head layout (ofrl_delta_create); the only allocation.

    backward=False reserves no memory for delta_backward, which is then refused."""

    def __init__(self, k_heads: int, v_heads: int, k_dim: int, v_dim: int, dtype: str = "bf16",
                 max_tokens: int = 16384, max_episodes: int = 1024, backward: bool = True):
        self._lib = _abi.load()
        self.shape = _abi.DeltaShape(k_heads, v_heads, k_dim, v_dim, DTYPE[dtype])
        self.k_heads, self.v_heads, self.k_dim, self.v_dim = k_heads, v_heads, k_dim, v_dim
        self.dtype = _TORCH_DTYPE[dtype]
        self.max_tokens, self.max_episodes, self.backward = max_tokens, max_episodes, bool(backward)
        self.shape_ref = C.byref(self.shape)
        self.device = torch.cuda.current_device()
        self.handle = None
        h = C.c_void_p()
        _abi.check("ofrl_delta_create", self._lib.ofrl_delta_create(
            C.byref(self.shape), max_tokens, max_episodes, int(self.backward), C.byref(h)))
        self.handle = h

    def close(self):
        if self.handle is not None and self.handle.value:
            _abi.check("ofrl_delta_destroy", self._lib.ofrl_delta_destroy(self.handle))
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def poll_status(self, stream=None):
        words = (C.c_int32 * _abi.STAT_WORDS)()
        _abi.check("ofrl_delta_poll_status", self._lib.ofrl_delta_poll_status(self.handle, _stream(stream), words))
        return {"bad_index": words[_abi.STAT_BAD_INDEX], "timeout": words[_abi.STAT_TIMEOUT]}

    def workspace_bytes(self) -> int:
        return int(self._lib.ofrl_delta_workspace_bytes(C.byref(self.shape), self.max_tokens, self.max_episodes,
                                                        int(self.backward)))

    def saved(self, tokens: int, episodes: int) -> torch.Tensor:
        """A buffer for the states that delta_forward hands to delta_backward."""
        n = int(self._lib.ofrl_delta_saved_bytes(C.byref(self.shape), tokens, episodes))
        if n < 0:
            raise ValueError(f"ofrl_delta_saved_bytes: invalid arguments (tokens={tokens}, episodes={episodes})")
        return torch.empty(max(n, 1), device="cuda", dtype=torch.uint8)


def _refuse(t, dtype, shape, name: str):
    """Raise for a tensor that is not a CUDA tensor of this type and shape."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


def _rows3(t: torch.Tensor, dtype, shape, name: str):
    """Address and row stride (elements) of a CUDA tensor [tokens, heads, channels] whose rows are dense."""
    if type(t) is not _TENSOR or t.dtype is not dtype or t.shape != shape or not t.is_cuda:
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or not t.is_cuda:
            _refuse(t, dtype, shape, name)
    s0, s1, s2 = t.stride()
    n, h, d = shape
    if n and (s2 != 1 and d > 1 or s1 != d and h > 1):
        raise ValueError(f"{name} must have dense rows (heads and channels contiguous within a token)")
    return t.data_ptr(), s0 if n > 1 else h * d


def _rows2(t: torch.Tensor, dtype, shape, name: str):
    """Address and row stride (elements) of a CUDA tensor [tokens, heads] whose rows are dense."""
    if type(t) is not _TENSOR or t.dtype is not dtype or t.shape != shape or not t.is_cuda:
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or not t.is_cuda:
            _refuse(t, dtype, shape, name)
    s0, s1 = t.stride()
    n, h = shape
    if n and s1 != 1 and h > 1:
        raise ValueError(f"{name} must have dense rows (heads contiguous within a token)")
    return t.data_ptr(), s0 if n > 1 else h


def _dense(t: Optional[torch.Tensor], dtype, shape, name: str):
    """Address of a contiguous CUDA tensor of this shape (0 for None)."""
    if t is None:
        return 0
    if type(t) is not _TENSOR or t.dtype is not dtype or t.shape != shape or not t.is_cuda:
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or not t.is_cuda:
            _refuse(t, dtype, shape, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)      # absent where torch has no CUDA


def _raw_stream(stream, device: int) -> int:
    return _current_stream(device) if stream is None else stream.cuda_stream


def _delta_tokens(ctx: DeltaRule, q, k, v, g, beta, scale):
    """The packed ofrl_delta_tokens, the token count and the three shapes."""
    dt = ctx.dtype
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        _refuse(q, dt, ("tokens", ctx.k_heads, ctx.k_dim), "q")
    n = q.shape[0]
    qk, vv, hv = (n, ctx.k_heads, ctx.k_dim), (n, ctx.v_heads, ctx.v_dim), (n, ctx.v_heads)
    q, qs = _rows3(q, dt, qk, "q")
    k, ks = _rows3(k, dt, qk, "k")
    v, vs = _rows3(v, dt, vv, "v")
    g, gs = _rows2(g, dt, hv, "g")
    beta, bs = _rows2(beta, dt, hv, "beta")
    return (_pack_tokens(q, k, v, g, beta, qs, ks, vs, gs, bs, n, ctx.k_dim ** -0.5 if scale is None else scale),
            n, qk, vv, hv)


_pack_tokens = struct.Struct(_abi.DELTA_TOKENS_FMT).pack
_pack_grads = struct.Struct(_abi.DELTA_GRADS_FMT).pack


def delta_forward(ctx: DeltaRule, q, k, v, g, beta, episode_ends, out, scale=None, init_state=None, final_state=None,
                  saved=None, stream=None):
    """The gated delta rule over packed episodes: q, k [tokens, k_heads, k_dim], v and out [tokens, v_heads, v_dim],
    g (log decay) and beta [tokens, v_heads] (out contiguous; the others may be slices with dense rows);
    episode_ends int32 [episodes].  scale: of the outputs (k_dim ** -0.5).  init_state, final_state: float32
    [episodes, v_heads, v_dim, k_dim].  saved: ctx.saved(tokens, episodes), filled for delta_backward."""
    t, n, _, vv, _ = _delta_tokens(ctx, q, k, v, g, beta, scale)
    ne = episode_ends.numel()
    state = (ne, ctx.v_heads, ctx.v_dim, ctx.k_dim)
    code = ctx._lib.ofrl_delta_forward(
        ctx.handle, t, _dense(episode_ends, I32, (ne,), "episode_ends"), ne,
        _dense(init_state, F32, state, "init_state"), _dense(out, ctx.dtype, vv, "out"),
        _dense(final_state, F32, state, "final_state"), _saved_ptr(ctx, saved, n, ne), _raw_stream(stream, ctx.device))
    if code != _abi.OK:
        _abi.check("ofrl_delta_forward", code)


def _saved_ptr(ctx: DeltaRule, saved, tokens: int, episodes: int):
    if saved is None:
        return 0
    need = ctx._lib.ofrl_delta_saved_bytes(ctx.shape_ref, tokens, episodes)
    if saved.numel() < need:
        raise ValueError(f"saved has {saved.numel()} bytes, {need} are needed: use ctx.saved(tokens, episodes)")
    return _dense(saved, torch.uint8, saved.shape, "saved")


def delta_backward(ctx: DeltaRule, q, k, v, g, beta, episode_ends, saved, dout, dq, dk, dv, dg, dbeta, scale=None,
                   d_final=None, d_init=None, stream=None):
    """Gradients of the delta_forward call that filled `saved`, with the same inputs: of out in dout (contiguous), of
    final_state in d_final (None: zero); written to dq, dk, dv, dg, dbeta (slices with dense rows) and d_init."""
    t, n, qk, vv, hv = _delta_tokens(ctx, q, k, v, g, beta, scale)
    ne = episode_ends.numel()
    if saved is None:
        raise TypeError("saved must be the buffer that delta_forward filled")
    dt = ctx.dtype
    state = (ne, ctx.v_heads, ctx.v_dim, ctx.k_dim)
    dq, qs = _rows3(dq, dt, qk, "dq")
    dk, ks = _rows3(dk, dt, qk, "dk")
    dv, vs = _rows3(dv, dt, vv, "dv")
    dg, gs = _rows2(dg, dt, hv, "dg")
    dbeta, bs = _rows2(dbeta, dt, hv, "dbeta")
    code = ctx._lib.ofrl_delta_backward(
        ctx.handle, t, _dense(episode_ends, I32, (ne,), "episode_ends"), ne, _saved_ptr(ctx, saved, n, ne),
        _dense(dout, dt, vv, "dout"), _dense(d_final, F32, state, "d_final"),
        _pack_grads(dq, dk, dv, dg, dbeta, qs, ks, vs, gs, bs), _dense(d_init, F32, state, "d_init"),
        _raw_stream(stream, ctx.device))
    if code != _abi.OK:
        _abi.check("ofrl_delta_backward", code)


def delta_step(ctx: DeltaRule, q, k, v, g, beta, state, out, scale=None, new_state=None, slots=None, stream=None):
    """One token for each environment: tensors as delta_forward's with tokens = environments; state float32 [slots,
    v_heads, v_dim, k_dim], updated in place or written to new_state (which shares no memory with it); slots: int32
    [tokens], the state of each token (None: token i has state i)."""
    t, n, _, vv, _ = _delta_tokens(ctx, q, k, v, g, beta, scale)
    ns = state.shape[0]
    shape = (ns, ctx.v_heads, ctx.v_dim, ctx.k_dim)
    at = _dense(state, F32, shape, "state")
    code = ctx._lib.ofrl_delta_step(
        ctx.handle, t, 0 if slots is None else _dense(slots, I32, (n,), "slots"), ns, at,
        at if new_state is None else _dense(new_state, F32, shape, "new_state"), _dense(out, ctx.dtype, vv, "out"),
        _raw_stream(stream, ctx.device))
    if code != _abi.OK:
        _abi.check("ofrl_delta_step", code)


# ---- state space blocks ----------------------------------------------------------------------------------------------

ACTIVATION = {"none": _abi.ACT_NONE, "silu": _abi.ACT_SILU}


class _Workspace:
    """A handle of the library with its device, closed at most once."""

    def _create(self, name: str, *args):
        self._lib = _abi.load()
        self._name = name
        self.handle = None
        self.device = torch.cuda.current_device()
        h = C.c_void_p()
        _abi.check(f"ofrl_{name}_create", getattr(self._lib, f"ofrl_{name}_create")(*args, C.byref(h)))
        self.handle = h

    def close(self):
        if self.handle is not None and self.handle.value:
            _abi.check(f"ofrl_{self._name}_destroy", getattr(self._lib, f"ofrl_{self._name}_destroy")(self.handle))
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _poll(self, stream=None):
        words = (C.c_int32 * _abi.STAT_WORDS)()
        name = f"ofrl_{self._name}_poll_status"
        _abi.check(name, getattr(self._lib, name)(self.handle, _stream(stream), words))
        return {"bad_index": words[_abi.STAT_BAD_INDEX]}


class CausalConv(_Workspace):
    """Workspace of the short causal convolution (ofrl_conv_create); the only allocation.

    channels: a multiple of 8; width: 2, 3 or 4 taps; activation: "none" or "silu".  backward=False reserves no
    memory for conv_backward, which is then refused."""

    def __init__(self, channels: int, width: int = 4, activation: str = "silu", dtype: str = "bf16",
                 max_tokens: int = 16384, max_episodes: int = 1024, backward: bool = True):
        self.shape = _abi.ConvShape(channels, width, ACTIVATION[activation], DTYPE[dtype])
        self.channels, self.width, self.activation = channels, width, activation
        self.dtype = _TORCH_DTYPE[dtype]
        self.max_tokens, self.max_episodes, self.backward = max_tokens, max_episodes, bool(backward)
        self._create("conv", C.byref(self.shape), max_tokens, max_episodes, int(self.backward))

    def poll_status(self, stream=None):
        return self._poll(stream)

    def workspace_bytes(self) -> int:
        return int(self._lib.ofrl_conv_workspace_bytes(C.byref(self.shape), self.max_tokens, self.max_episodes,
                                                       int(self.backward)))


class SelectiveScan(_Workspace):
    """Workspace of the selective scan (ofrl_scan_create); the only allocation.

    state_dim: 4 to 64, a multiple of 4; groups of channels share B and C; channels / groups: a multiple of 8.
    softplus=False takes dt + dt_bias as it is.  backward=False reserves no memory for scan_backward, which is then
    refused."""

    def __init__(self, channels: int, state_dim: int = 16, groups: int = 1, dtype: str = "bf16", softplus: bool = True,
                 max_tokens: int = 16384, max_episodes: int = 1024, backward: bool = True):
        self.shape = _abi.ScanShape(channels, state_dim, groups, DTYPE[dtype], int(bool(softplus)))
        self.channels, self.state_dim, self.groups = channels, state_dim, groups
        self.dtype = _TORCH_DTYPE[dtype]
        self.max_tokens, self.max_episodes, self.backward = max_tokens, max_episodes, bool(backward)
        self._create("scan", C.byref(self.shape), max_tokens, max_episodes, int(self.backward))

    def poll_status(self, stream=None):
        return self._poll(stream)

    def workspace_bytes(self) -> int:
        return int(self._lib.ofrl_scan_workspace_bytes(C.byref(self.shape), self.max_tokens, self.max_episodes,
                                                       int(self.backward)))

    def saved(self, tokens: int) -> torch.Tensor:
        """A buffer for the states that scan_forward hands to scan_backward."""
        n = int(self._lib.ofrl_scan_saved_bytes(C.byref(self.shape), tokens))
        if n < 0:
            raise ValueError(f"ofrl_scan_saved_bytes: invalid arguments (tokens={tokens})")
        return torch.empty(max(n, 1), device=f"cuda:{self.device}", dtype=torch.uint8)


class BlockNorm(_Workspace):
    """Workspace of the gated norm and the residual norm (ofrl_norm_create); the only allocation.

    Each of `groups` equal groups of channels is normed by itself.  residual_dtype: the residual stream's type, "fp32"
    or dtype (the default).  backward=False reserves no memory for the gradients, which are then refused.  Two backward
    calls with one workspace must not overlap on the GPU: it holds their parts of the weights' gradients."""

    def __init__(self, channels: int, groups: int = 1, dtype: str = "bf16", residual_dtype: Optional[str] = None,
                 backward: bool = True):
        residual_dtype = dtype if residual_dtype is None else residual_dtype
        self.shape = _abi.NormShape(channels, groups, DTYPE[dtype], DTYPE[residual_dtype])
        self.channels, self.groups = channels, groups
        self.dtype, self.residual_dtype = _TORCH_DTYPE[dtype], _TORCH_DTYPE[residual_dtype]
        self.backward = bool(backward)
        self._create("norm", C.byref(self.shape), int(self.backward))

    def workspace_bytes(self) -> int:
        return int(self._lib.ofrl_norm_workspace_bytes(C.byref(self.shape), int(self.backward)))


def _open_ctx(ctx, kind):
    """The handle of a workspace of this class that is open."""
    if not isinstance(ctx, kind):
        raise TypeError(f"ctx must be a {kind.__name__}")
    if ctx.handle is None:
        raise ValueError(f"the {kind.__name__} is closed")
    return ctx.handle


def _refuse_at(t, dtype, shape, name, device):
    """Raise unless this is a CUDA tensor of this type and shape on the workspace's device: a kernel would follow its
    address there."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or not t.is_cuda:
        _refuse(t, dtype, shape, name)
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, where the workspace is, got {t.device}")


def _rows3_at(t, dtype, shape, name, device):
    """Address and row stride (elements) of a tensor [tokens, groups, states] on this device whose rows are dense."""
    if type(t) is not _TENSOR or t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        _refuse_at(t, dtype, shape, name, device)
    s0, s1, s2 = t.stride()
    n, h, d = shape
    if n and (s2 != 1 and d > 1 or s1 != d and h > 1):
        raise ValueError(f"{name} must have dense rows (groups and states contiguous within a token)")
    return t.data_ptr(), s0 if n > 1 else h * d


def _rows2_at(t, dtype, shape, name, device):
    """Address and row stride (elements) of a tensor [tokens, channels] on this device whose rows are dense."""
    if type(t) is not _TENSOR or t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        _refuse_at(t, dtype, shape, name, device)
    s0, s1 = t.stride()
    n, h = shape
    if n and s1 != 1 and h > 1:
        raise ValueError(f"{name} must have dense rows (channels contiguous within a token)")
    return t.data_ptr(), s0 if n > 1 else h


def _dense_at(t, dtype, shape, name, device):
    """Address of a contiguous tensor of this shape on this device (0 for None)."""
    if t is None:
        return 0
    if type(t) is not _TENSOR or t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        _refuse_at(t, dtype, shape, name, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _tokens_of(x, channels: int, dtype, name: str) -> int:
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        _refuse(x, dtype, ("tokens", channels), name)
    return x.shape[0]


_pack_conv_tokens = struct.Struct(_abi.CONV_TOKENS_FMT).pack
_pack_conv_grads = struct.Struct(_abi.CONV_GRADS_FMT).pack
_pack_scan_tokens = struct.Struct(_abi.SCAN_TOKENS_FMT).pack
_pack_scan_grads = struct.Struct(_abi.SCAN_GRADS_FMT).pack
_pack_gated_rows = struct.Struct(_abi.GATED_ROWS_FMT).pack
_pack_residual_rows = struct.Struct(_abi.RESIDUAL_ROWS_FMT).pack


def _conv_tokens(ctx: CausalConv, x, weight, bias):
    """The packed ofrl_conv_tokens and the shape of x."""
    dev = ctx.device
    d = ctx.channels
    rows = (_tokens_of(x, d, ctx.dtype, "x"), d)
    x, xs = _rows2_at(x, ctx.dtype, rows, "x", dev)
    w = _dense_at(weight, F32, (d, ctx.width), "weight", dev)
    return _pack_conv_tokens(x, w, _dense_at(bias, F32, (d,), "bias", dev), xs, rows[0]), rows


def conv_forward(ctx: CausalConv, x, weight, episode_ends, out, bias=None, init_state=None, final_state=None, stream=None):
    """out = act(causal convolution of x) over packed episodes: x, out [tokens, channels] (may be slices with dense
    rows), weight float32 [channels, width] (the last tap takes the token itself), bias float32 [channels];
    episode_ends int32 [episodes].  init_state, final_state: [episodes, channels, width - 1] of x's type, the inputs
    before an episode and its last ones (two buffers)."""
    handle = _open_ctx(ctx, CausalConv)
    dev = ctx.device
    t, rows = _conv_tokens(ctx, x, weight, bias)
    ne = episode_ends.numel()
    state = (ne, ctx.channels, ctx.width - 1)
    o, os = _rows2_at(out, ctx.dtype, rows, "out", dev)
    init = _dense_at(init_state, ctx.dtype, state, "init_state", dev)
    final = _dense_at(final_state, ctx.dtype, state, "final_state", dev)
    ends = _dense_at(episode_ends, I32, (ne,), "episode_ends", dev)
    code = ctx._lib.ofrl_conv_forward(handle, t, ends, ne, init, o, os, final, _raw_stream(stream, dev))
    if code != _abi.OK:
        _abi.check("ofrl_conv_forward", code)


def conv_backward(ctx: CausalConv, x, weight, episode_ends, dout, dx, dweight, bias=None, dbias=None, init_state=None,
                  d_final=None, d_init=None, stream=None):
    """Gradients of the conv_forward call with the same inputs: of out in dout, of final_state in d_final (of x's type;
    None: zero); written to dx, dweight, dbias and d_init (float32; the last two may be None)."""
    handle = _open_ctx(ctx, CausalConv)
    dev = ctx.device
    t, rows = _conv_tokens(ctx, x, weight, bias)
    ne, d = episode_ends.numel(), ctx.channels
    state = (ne, d, ctx.width - 1)
    g, gs = _rows2_at(dout, ctx.dtype, rows, "dout", dev)
    dxp, xs = _rows2_at(dx, ctx.dtype, rows, "dx", dev)
    if dweight is None:
        raise TypeError("dweight must be a CUDA tensor")
    init = _dense_at(init_state, ctx.dtype, state, "init_state", dev)
    dfin = _dense_at(d_final, ctx.dtype, state, "d_final", dev)
    dini, ends = _dense_at(d_init, F32, state, "d_init", dev), _dense_at(episode_ends, I32, (ne,), "episode_ends", dev)
    dw = _dense_at(dweight, F32, (d, ctx.width), "dweight", dev)
    grads = _pack_conv_grads(dxp, dw, _dense_at(dbias, F32, (d,), "dbias", dev), xs)
    code = ctx._lib.ofrl_conv_backward(handle, t, ends, ne, init, g, gs, dfin, grads, dini, _raw_stream(stream, dev))
    if code != _abi.OK:
        _abi.check("ofrl_conv_backward", code)


def _state_pair(state, new_state, dtype, tail, dev):
    """Addresses of a step's states and how many slots they have."""
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        _refuse(state, dtype, ("slots", *tail), "state")
    shape = (state.shape[0], *tail)
    at = _dense_at(state, dtype, shape, "state", dev)
    return at, at if new_state is None else _dense_at(new_state, dtype, shape, "new_state", dev), shape[0]


def conv_step(ctx: CausalConv, x, weight, state, out, bias=None, new_state=None, slots=None, stream=None):
    """One token for each environment: tensors as conv_forward's with tokens = environments; state [slots, channels,
    width - 1], updated in place or written to new_state (which shares no memory with it); slots: int32 [tokens], the
    state of each token (None: token i has state i)."""
    handle = _open_ctx(ctx, CausalConv)
    dev = ctx.device
    t, rows = _conv_tokens(ctx, x, weight, bias)
    at, to, ns = _state_pair(state, new_state, ctx.dtype, (ctx.channels, ctx.width - 1), dev)
    o, os = _rows2_at(out, ctx.dtype, rows, "out", dev)
    slot_idx = _dense_at(slots, I32, (rows[0],), "slots", dev)
    code = ctx._lib.ofrl_conv_step(handle, t, slot_idx, ns, at, to, o, os, _raw_stream(stream, dev))
    if code != _abi.OK:
        _abi.check("ofrl_conv_step", code)


def _scan_tokens(ctx: SelectiveScan, x, dt, A, B, C_, D, z, dt_bias):
    """The packed ofrl_scan_tokens and the shapes of x and of B."""
    dev = ctx.device
    d, n, ty = ctx.channels, ctx.state_dim, ctx.dtype
    rows = (_tokens_of(x, d, ty, "x"), d)
    bc = (rows[0], ctx.groups, n)
    x, xs = _rows2_at(x, ty, rows, "x", dev)
    dt, ds = _rows2_at(dt, ty, rows, "dt", dev)
    B, bs = _rows3_at(B, ty, bc, "B", dev)
    C_, cs = _rows3_at(C_, ty, bc, "C", dev)
    z, zs = (0, 0) if z is None else _rows2_at(z, ty, rows, "z", dev)
    if A is None:
        raise TypeError("A must be a CUDA tensor")
    return _pack_scan_tokens(x, dt, B, C_, z, _dense_at(A, F32, (d, n), "A", dev), _dense_at(D, F32, (d,), "D", dev),
                             _dense_at(dt_bias, F32, (d,), "dt_bias", dev), xs, ds, bs, cs, zs, rows[0]), rows, bc


def _scan_saved(ctx: SelectiveScan, saved, tokens: int):
    if saved is None:
        return 0
    need = ctx._lib.ofrl_scan_saved_bytes(C.byref(ctx.shape), tokens)
    if saved.numel() < need:
        raise ValueError(f"saved has {saved.numel()} bytes, {need} are needed: use ctx.saved(tokens)")
    return _dense_at(saved, torch.uint8, saved.shape, "saved", ctx.device)


def scan_forward(ctx: SelectiveScan, x, dt, A, B, C, episode_ends, out, D=None, z=None, dt_bias=None, init_state=None,
                 final_state=None, saved=None, stream=None):
    """The selective scan over packed episodes: x, dt, z, out [tokens, channels], B, C [tokens, groups, state_dim] (all
    may be slices with dense rows); A float32 [channels, state_dim] (negative), D and dt_bias float32 [channels];
    episode_ends int32 [episodes].  init_state, final_state: float32 [episodes, channels, state_dim] (two buffers).
    saved: ctx.saved(tokens), filled for scan_backward."""
    handle = _open_ctx(ctx, SelectiveScan)
    dev = ctx.device
    t, rows, _ = _scan_tokens(ctx, x, dt, A, B, C, D, z, dt_bias)
    ne = episode_ends.numel()
    state = (ne, ctx.channels, ctx.state_dim)
    o, os = _rows2_at(out, ctx.dtype, rows, "out", dev)
    init = _dense_at(init_state, F32, state, "init_state", dev)
    final = _dense_at(final_state, F32, state, "final_state", dev)
    ends, kept = _dense_at(episode_ends, I32, (ne,), "episode_ends", dev), _scan_saved(ctx, saved, rows[0])
    code = ctx._lib.ofrl_scan_forward(handle, t, ends, ne, init, o, os, final, kept, _raw_stream(stream, dev))
    if code != _abi.OK:
        _abi.check("ofrl_scan_forward", code)


def scan_backward(ctx: SelectiveScan, x, dt, A, B, C, episode_ends, saved, dout, dx, ddt, dA, dB, dC, D=None, z=None,
                  dt_bias=None, dD=None, dz=None, ddt_bias=None, init_state=None, d_final=None, d_init=None, stream=None):
    """Gradients of the scan_forward call that filled `saved`, with the same inputs: of out in dout, of final_state in
    d_final (None: zero); written to dx, ddt, dB, dC, dz (given where z is; slices with dense rows), and to dA, dD,
    ddt_bias and d_init (float32; the last three may be None)."""
    handle = _open_ctx(ctx, SelectiveScan)
    dev = ctx.device
    t, rows, bc = _scan_tokens(ctx, x, dt, A, B, C, D, z, dt_bias)
    if saved is None:
        raise TypeError("saved must be the buffer that scan_forward filled")
    if dA is None:
        raise TypeError("dA must be a CUDA tensor")
    ne, d, ty = episode_ends.numel(), ctx.channels, ctx.dtype
    state = (ne, d, ctx.state_dim)
    g, gs = _rows2_at(dout, ty, rows, "dout", dev)
    dxp, xs = _rows2_at(dx, ty, rows, "dx", dev)
    ddtp, ds = _rows2_at(ddt, ty, rows, "ddt", dev)
    dBp, bs = _rows3_at(dB, ty, bc, "dB", dev)
    dCp, cs = _rows3_at(dC, ty, bc, "dC", dev)
    dzp, zs = (0, 0) if dz is None else _rows2_at(dz, ty, rows, "dz", dev)
    init, dfin = _dense_at(init_state, F32, state, "init_state", dev), _dense_at(d_final, F32, state, "d_final", dev)
    dini, ends = _dense_at(d_init, F32, state, "d_init", dev), _dense_at(episode_ends, I32, (ne,), "episode_ends", dev)
    kept = _scan_saved(ctx, saved, rows[0])
    dAp, dDp = _dense_at(dA, F32, (d, ctx.state_dim), "dA", dev), _dense_at(dD, F32, (d,), "dD", dev)
    grads = _pack_scan_grads(dxp, ddtp, dBp, dCp, dzp, dAp, dDp, _dense_at(ddt_bias, F32, (d,), "ddt_bias", dev), xs, ds, bs,
                             cs, zs)
    code = ctx._lib.ofrl_scan_backward(handle, t, ends, ne, init, kept, g, gs, dfin, grads, dini,
                                       _raw_stream(stream, dev))
    if code != _abi.OK:
        _abi.check("ofrl_scan_backward", code)


def scan_step(ctx: SelectiveScan, x, dt, A, B, C, state, out, D=None, z=None, dt_bias=None, new_state=None, slots=None,
              stream=None):
    """One token for each environment: tensors as scan_forward's with tokens = environments; state float32 [slots,
    channels, state_dim], updated in place or written to new_state (which shares no memory with it); slots: int32
    [tokens], the state of each token (None: token i has state i)."""
    handle = _open_ctx(ctx, SelectiveScan)
    dev = ctx.device
    t, rows, _ = _scan_tokens(ctx, x, dt, A, B, C, D, z, dt_bias)
    at, to, ns = _state_pair(state, new_state, F32, (ctx.channels, ctx.state_dim), dev)
    o, os = _rows2_at(out, ctx.dtype, rows, "out", dev)
    slot_idx = _dense_at(slots, I32, (rows[0],), "slots", dev)
    code = ctx._lib.ofrl_scan_step(handle, t, slot_idx, ns, at, to, o, os, _raw_stream(stream, dev))
    if code != _abi.OK:
        _abi.check("ofrl_scan_step", code)


def _norm_weight(ctx: BlockNorm, weight, name="weight"):
    if weight is None:
        raise TypeError(f"{name} must be a CUDA tensor")
    return _dense_at(weight, F32, (ctx.channels,), name, ctx.device)


def _gated_rows(ctx: BlockNorm, x, z, weight, eps, gate_first):
    dev = ctx.device
    rows = (_tokens_of(x, ctx.channels, ctx.dtype, "x"), ctx.channels)
    x, xs = _rows2_at(x, ctx.dtype, rows, "x", dev)
    z, zs = _rows2_at(z, ctx.dtype, rows, "z", dev)
    return _pack_gated_rows(x, z, _norm_weight(ctx, weight), xs, zs, rows[0], eps, bool(gate_first)), rows


def gated_norm(ctx: BlockNorm, x, z, weight, out, eps: float = 1e-5, gate_first: bool = False, stream=None):
    """out = weight x / rms(x) silu(z), or the norm of x silu(z) (gate_first), over each group of channels: x, z, out
    [rows, channels] (may be slices with dense rows; out may be x), weight float32 [channels]."""
    handle = _open_ctx(ctx, BlockNorm)
    dev = ctx.device
    t, rows = _gated_rows(ctx, x, z, weight, eps, gate_first)
    o, os = _rows2_at(out, ctx.dtype, rows, "out", dev)
    code = ctx._lib.ofrl_gated_norm(handle, t, o, os, _raw_stream(stream, dev))
    if code != _abi.OK:
        _abi.check("ofrl_gated_norm", code)


def gated_norm_backward(ctx: BlockNorm, x, z, weight, dout, dx, dz, dweight, eps: float = 1e-5, gate_first: bool = False,
                        stream=None):
    """Gradients of the gated_norm call with the same inputs, written to dx, dz (slices with dense rows) and dweight."""
    handle = _open_ctx(ctx, BlockNorm)
    dev = ctx.device
    t, rows = _gated_rows(ctx, x, z, weight, eps, gate_first)
    g, gs = _rows2_at(dout, ctx.dtype, rows, "dout", dev)
    dxp, xs = _rows2_at(dx, ctx.dtype, rows, "dx", dev)
    dzp, zs = _rows2_at(dz, ctx.dtype, rows, "dz", dev)
    dw = _norm_weight(ctx, dweight, "dweight")
    code = ctx._lib.ofrl_gated_norm_backward(handle, t, g, gs, dxp, xs, dzp, zs, dw, _raw_stream(stream, dev))
    if code != _abi.OK:
        _abi.check("ofrl_gated_norm_backward", code)


def _residual_rows(ctx: BlockNorm, x, residual, scale, weight, eps):
    dev = ctx.device
    rows = (_tokens_of(x, ctx.channels, ctx.dtype, "x"), ctx.channels)
    x, xs = _rows2_at(x, ctx.dtype, rows, "x", dev)
    residual, rs = _rows2_at(residual, ctx.residual_dtype, rows, "residual", dev)
    scale = _dense_at(scale, F32, (ctx.channels,), "scale", dev)
    return _pack_residual_rows(x, residual, scale, _norm_weight(ctx, weight), xs, rs, rows[0], eps), rows


def residual_norm(ctx: BlockNorm, x, residual, weight, residual_out, out, scale=None, eps: float = 1e-5, stream=None):
    """residual_out = residual + scale x and out = weight residual_out / rms(residual_out) (of the sum before it is
    rounded to its type): x, out [rows, channels], residual, residual_out of the residual's type (all may be slices
    with dense rows; residual_out may be residual, out may be x), scale (None: one) and weight float32 [channels]."""
    handle = _open_ctx(ctx, BlockNorm)
    dev = ctx.device
    t, rows = _residual_rows(ctx, x, residual, scale, weight, eps)
    r, rs = _rows2_at(residual_out, ctx.residual_dtype, rows, "residual_out", dev)
    o, os = _rows2_at(out, ctx.dtype, rows, "out", dev)
    code = ctx._lib.ofrl_residual_norm(handle, t, r, rs, o, os, _raw_stream(stream, dev))
    if code != _abi.OK:
        _abi.check("ofrl_residual_norm", code)


def residual_norm_backward(ctx: BlockNorm, x, residual, weight, dout, dx, dresidual, dweight, scale=None, dscale=None,
                           d_residual_out=None, eps: float = 1e-5, stream=None):
    """Gradients of the residual_norm call with the same inputs: of out in dout, of residual_out in d_residual_out
    (None: zero); written to dx, dresidual (slices with dense rows), dweight, and dscale (given where scale is)."""
    handle = _open_ctx(ctx, BlockNorm)
    dev = ctx.device
    t, rows = _residual_rows(ctx, x, residual, scale, weight, eps)
    g, gs = _rows2_at(dout, ctx.dtype, rows, "dout", dev)
    dxp, xs = _rows2_at(dx, ctx.dtype, rows, "dx", dev)
    dr, drs = _rows2_at(dresidual, ctx.residual_dtype, rows, "dresidual", dev)
    do = dos = 0
    if d_residual_out is not None:
        do, dos = _rows2_at(d_residual_out, ctx.residual_dtype, rows, "d_residual_out", dev)
    dw, dsc = _norm_weight(ctx, dweight, "dweight"), _dense_at(dscale, F32, (ctx.channels,), "dscale", dev)
    code = ctx._lib.ofrl_residual_norm_backward(handle, t, g, gs, do, dos, dxp, xs, dr, drs, dw, dsc,
                                                _raw_stream(stream, dev))
    if code != _abi.OK:
        _abi.check("ofrl_residual_norm_backward", code)


# ---- gradients kept in many tensors --------------------------------------------------------------------------------


class TensorList:
    """A list of contiguous float32 or bfloat16 CUDA tensors (ofrl_tensors_create): what global_norm and
    global_norm_clip read and write.  It holds the tensors; their memory must stay where it is."""

    def __init__(self, tensors: Sequence[torch.Tensor]):
        self._lib = _abi.load()
        self.handle = None
        self.tensors = list(tensors)
        self.device = torch.cuda.current_device()
        n = len(self.tensors)
        ptrs, sizes, dtypes = (C.c_void_p * max(n, 1))(), (C.c_int64 * max(n, 1))(), (C.c_int32 * max(n, 1))()
        codes = {F32: _abi.DTYPE_F32, BF16: _abi.DTYPE_BF16}
        for i, t in enumerate(self.tensors):
            p = _ptr(t, None, "tensor")
            if t.dtype not in codes:
                raise TypeError(f"tensor {i} must be float32 or bfloat16, got {t.dtype}")
            ptrs[i], sizes[i], dtypes[i] = p.value, t.numel(), codes[t.dtype]
        h = C.c_void_p()
        _abi.check("ofrl_tensors_create", self._lib.ofrl_tensors_create(ptrs, sizes, dtypes, n, C.byref(h)))
        self.handle = h

    def close(self):
        if self.handle is not None and self.handle.value:
            _abi.check("ofrl_tensors_destroy", self._lib.ofrl_tensors_destroy(self.handle))
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _open(tensors: TensorList, name: str):
    """The handle of a list that is open (NULL would say that there is none)."""
    if not isinstance(tensors, TensorList):
        raise TypeError(f"{name} must be a TensorList")
    if tensors.handle is None:
        raise ValueError(f"{name} is closed")
    return tensors.handle


def global_norm(tensors: TensorList, norm_out, stream=None):
    """norm_out[0] = the 2-norm over all elements of all tensors (adam_step's grad_norm)."""
    code = tensors._lib.ofrl_global_norm(_open(tensors, "tensors"), _dense(norm_out, F32, (1,), "norm_out"),
                                         _raw_stream(stream, tensors.device))
    if code != _abi.OK:
        _abi.check("ofrl_global_norm", code)


def global_norm_clip(tensors: TensorList, max_norm: float, norm_out, out: Optional[TensorList] = None, stream=None):
    """global_norm, then every element times min(1, max_norm / norm), in place or into the tensors of `out`."""
    code = tensors._lib.ofrl_global_norm_clip(
        _open(tensors, "tensors"), max_norm, _dense(norm_out, F32, (1,), "norm_out"),
        None if out is None else _open(out, "out"),
        _raw_stream(stream, tensors.device))
    if code != _abi.OK:
        _abi.check("ofrl_global_norm_clip", code)


def train_step_kernels(ctx: Context, batch: Batch, rows: int, n_nets: int = 1) -> int:
    """Kernel launches one train_step makes for this batch (4, or 3 when the reduce and Adam run as one launch)."""
    b = batch.c()
    return int(ctx._lib.ofrl_train_step_kernels(ctx.handle, C.byref(b), rows, n_nets))


def profile_begin(ctx: Context, max_steps: int):
    _abi.check("ofrl_profile_begin", ctx._lib.ofrl_profile_begin(ctx.handle, max_steps))


def profile_end(ctx: Context):
    """Per-phase device milliseconds summed over the profiled steps, and the step count."""
    ms = (C.c_float * len(_abi.PHASES))()
    n = C.c_int32()
    _abi.check("ofrl_profile_end", ctx._lib.ofrl_profile_end(ctx.handle, ms, C.byref(n)))
    return dict(zip(_abi.PHASES, list(ms))), int(n.value)
