"""AdamW over many tensors at once, with moments in 32 or 8 bits, and the
gradients' norm and clipping factor (libgq_step.so, ``include/gq_step.h``).

They take what ``ddp.global_qsgd_hook`` leaves in the gradients.  A moment in
8 bits (``Moment8``) is one byte a value and a power of two for each 128: e4m3
for the first, 5 exponent and 3 mantissa bits for the second, which is never
negative.  Both are rounded at random without bias, with the compressor's
Philox uniforms; to nearest, a second moment that decays by a thousandth a
step would never move.  A bf16 parameter may be rounded at random too, so that
updates below its last place count in expectation.

``gqs_*`` are the C entry points on lists of device tensors, in place, on
torch's current stream or a given one, with no synchronization.  ``AdamW`` is
the optimizer of torch's interface.
"""
from __future__ import annotations

import itertools
import operator
import struct

import torch
from torch.autograd.graph import increment_version

from ._step import CAdamWArgs, check, lib
from .train import _current, _dtype, _Elsewhere, _elsewhere, _mix_seed

_E4M3 = torch.float8_e4m3fn


class Moment8:
    """A moment of a tensor of n elements in 8 bits: ``codes`` [128 G]
    (float8_e4m3fn for a first moment, uint8 for a second) and ``exps`` uint8
    [G], G = ceil(n / 128)."""

    __slots__ = ("codes", "exps", "n")

    def __init__(self, codes: torch.Tensor, exps: torch.Tensor, n: int):
        self.codes, self.exps, self.n = codes, exps, int(n)

    @classmethod
    def zeros(cls, n: int, device, second: bool) -> "Moment8":
        blocks = (int(n) + 127) // 128
        codes = torch.zeros(128 * blocks, dtype=torch.uint8, device=device)
        return cls(codes if second else codes.view(_E4M3),
                   torch.full((blocks,), 19 if second else 10, dtype=torch.uint8, device=device),
                   n)

    @property
    def second(self) -> bool:
        return self.codes.dtype == torch.uint8

    def __repr__(self):
        return f"Moment8({self.n}, {'second' if self.second else 'first'}, {self.codes.device})"


# Lists of a hundred tensors and more are looked over in a few microseconds:
# by maps of C functions, not tensor by tensor.
_dtype_of, _index = operator.attrgetter("dtype"), torch.Tensor.get_device
_numel, _data_ptr = torch.Tensor.numel, torch.Tensor.data_ptr
_device, _sparse = operator.attrgetter("device"), operator.attrgetter("is_sparse")
_codes, _exps, _count = map(operator.attrgetter, ("codes", "exps", "n"))


def _arrays(tensors, name: str, device, dtype=None):
    """(dtype, sizes, addresses) of contiguous device tensors of one dtype."""
    if not all(issubclass(kind, torch.Tensor) for kind in set(map(type, tensors))):
        raise ValueError(f"{name} must be device tensors")
    if set(map(_index, tensors)) != {device.index}:
        raise ValueError(f"{name} must be on {device}, got {sorted({str(t.device) for t in tensors})}")
    if not all(map(torch.Tensor.is_contiguous, tensors)):
        raise ValueError(f"{name} must be contiguous")
    types = set(map(_dtype_of, tensors))
    if len(types) > 1 or (dtype is not None and types != {dtype}):
        want = "one dtype" if dtype is None else str(dtype)
        raise TypeError(f"{name} must have {want}, got {sorted(map(str, types))}")
    return types.pop(), list(map(_numel, tensors)), list(map(_data_ptr, tensors))


def _moments(moments, name: str, sizes, device, second: bool):
    """(bits, codes or values, exps) of a list of moments."""
    if len(moments) != len(sizes):
        raise ValueError(f"{len(moments)} {name}, {len(sizes)} tensors")
    kinds = set(map(type, moments))
    if Moment8 not in kinds:
        _, counts, at = _arrays(moments, name, device, torch.float32)
        if counts != sizes:
            raise ValueError(f"{name} must have their parameters' sizes")
        return 32, at, itertools.repeat(0)
    if len(kinds) > 1:
        raise TypeError(f"{name} must be all Moment8 or all tensors")
    if list(map(_count, moments)) != sizes:
        raise ValueError(f"{name} must have their parameters' sizes")
    kind = torch.uint8 if second else _E4M3
    _, counts, codes = _arrays(list(map(_codes, moments)), f"{name}' codes", device, kind)
    _, groups, exps = _arrays(list(map(_exps, moments)), f"{name}' exps", device, torch.uint8)
    blocks = [(n + 127) >> 7 for n in sizes]
    if groups != blocks or counts != [b << 7 for b in blocks]:
        raise ValueError(f"{name} must hold a code for each of 128 G elements and G exps")
    return 8, codes, exps


def _list(*columns) -> bytes:
    """The C array of tensors whose seven columns these are."""
    words = list(itertools.chain.from_iterable(zip(*columns)))
    return struct.pack(f"{len(words)}Q", *words)


def _scalar(t, name: str, dtype, device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != dtype or t.numel() != 1:
        raise ValueError(f"{name} must be one {dtype} on {device}")
    return t.data_ptr()


def _tensors_of(*lists):
    held = []
    for given in lists:
        for t in given if isinstance(given, (list, tuple)) else (given,):
            held.extend((t.codes, t.exps) if isinstance(t, Moment8) else (t,))
    return held


def _device_of(tensors, name: str):
    first = tensors[0]
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        raise ValueError(f"{name} must be device tensors")
    return first.device


def gqs_adamw(params, grads, exp_avgs, exp_avg_sqs, *, step, lr, betas=(0.9, 0.999),
              eps: float = 1e-8, weight_decay: float = 1e-2, scale=None, seed=None,
              random=None, stream=None) -> None:
    """One AdamW step, in place, over lists of tensors: params of one dtype
    and grads of one dtype (fp32 or bf16 each), moments as fp32 tensors or
    Moment8, all contiguous on one device, no two overlapping.

    scale: a device float, the gradients' factor.  step counts from 1; it and
    lr may be device tensors (int64 and float32, one element), which a
    captured graph reads at every replay.  A `seed` is needed with Moment8; a
    bf16 parameter is rounded at random where one is given, unless `random` is
    False, and to nearest otherwise.  Calls of one step with one seed share
    random numbers between tensors of the same number in their lists: give
    each list its own.

    To autograd the params are changed in place, as by torch's own operations."""
    params, grads = list(params), list(grads)
    exp_avgs, exp_avg_sqs = list(exp_avgs), list(exp_avg_sqs)
    if len(params) != len(grads):
        raise ValueError(f"{len(params)} params, {len(grads)} grads")
    if not params:
        return
    device = _device_of(params, "params")
    if _elsewhere(device, stream):
        with _Elsewhere(device, stream, _tensors_of(params, grads, exp_avgs, exp_avg_sqs, scale,
                                                    step, lr)):
            return gqs_adamw(params, grads, exp_avgs, exp_avg_sqs, step=step, lr=lr, betas=betas,
                             eps=eps, weight_decay=weight_decay, scale=scale, seed=seed,
                             random=random)
    p_type, sizes, p_at = _arrays(params, "params", device)
    g_type, g_sizes, g_at = _arrays(grads, "grads", device)
    if g_sizes != sizes:
        raise ValueError("grads must have their parameters' sizes")
    bits, m_at, m_exps = _moments(exp_avgs, "exp_avgs", sizes, device, False)
    v_bits, v_at, v_exps = _moments(exp_avg_sqs, "exp_avg_sqs", sizes, device, True)
    if bits != v_bits:
        raise TypeError("exp_avgs and exp_avg_sqs must be both Moment8 or both tensors")
    if bits == 8 and seed is None:
        raise ValueError("moments in 8 bits are rounded at random: a seed is needed")
    if random and seed is None:
        raise ValueError("random rounding needs a seed")
    args = CAdamWArgs(0.0, betas[0], betas[1], eps, weight_decay, 0,
                      _scalar(scale, "scale", torch.float32, device), None, None,
                      0 if seed is None else int(seed) & 0xFFFFFFFFFFFFFFFF,
                      seed is not None if random is None else bool(random), bits)
    workspace = None
    if isinstance(lr, torch.Tensor):
        args.lr_device = _scalar(lr, "lr", torch.float32, device)
    else:
        args.lr = lr
    if isinstance(step, torch.Tensor):
        args.step_device = _scalar(step, "step", torch.int64, device)
    else:
        args.step = step
    if args.lr_device or args.step_device:
        workspace = torch.empty(16, dtype=torch.uint8, device=device)
    check(lib().gqs_adamw(_list(p_at, g_at, m_at, v_at, m_exps, v_exps, sizes), len(sizes),
                          _dtype(p_type, "params"), _dtype(g_type, "grads"), args,
                          None if workspace is None else workspace.data_ptr(), 16,
                          _current(device)))
    increment_version(params)  # a graph that saved one is refused its backward pass


def gqs_moment8_restore(moment: Moment8, dtype=torch.bfloat16, *, stream=None) -> torch.Tensor:
    """The values a moment stands for, [n] (exact in either dtype)."""
    dt = _dtype(dtype, "dtype")
    if not isinstance(moment, Moment8) or not moment.codes.is_cuda:
        raise ValueError("moment must be a Moment8 on a device")
    device = moment.codes.device
    if _elsewhere(device, stream):
        with _Elsewhere(device, stream, _tensors_of(moment)):
            return gqs_moment8_restore(moment, dtype)
    second = moment.second
    _, (codes,), (exps,) = _moments([moment], "moment", [moment.n], device, second)
    out = torch.empty(moment.n, dtype=dtype, device=device)
    check(lib().gqs_moment8_restore(codes, exps, moment.n, second, dt, out.data_ptr(),
                                    _current(device)))
    return out


def gqs_grad_norm(grads, *, max_norm=None, stream=None):
    """(norm, scale) over a list of contiguous gradients of one dtype on one
    device, both fp32 device tensors of one element: their 2-norm, summed in
    fp64, and with `max_norm` the factor min(1, max_norm / (norm + 1e-6)) that
    clips them (None without), which gqs_adamw reads where it is."""
    grads = list(grads)
    if not grads:
        raise ValueError("grads is empty")
    device = _device_of(grads, "grads")
    if _elsewhere(device, stream):
        with _Elsewhere(device, stream, grads):
            return gqs_grad_norm(grads, max_norm=max_norm)
    kind, sizes, at = _arrays(grads, "grads", device)
    none = itertools.repeat(0)
    tensors = _list(none, at, none, none, none, none, sizes)
    need = lib().gqs_grad_norm_workspace_bytes(tensors, len(sizes))
    workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    out = torch.empty(2, dtype=torch.float32, device=device)
    norm, scale = out[0], out[1] if max_norm is not None else None
    check(lib().gqs_grad_norm(tensors, len(sizes), _dtype(kind, "grads"),
                              0.0 if max_norm is None else max_norm, norm.data_ptr(),
                              None if scale is None else scale.data_ptr(), workspace.data_ptr(),
                              max(need, 0), _current(device)))
    return norm, scale


# ---------------------------------------------------------------------------
# the optimizer

def _order(p):
    """The order of p's dimensions in which its elements lie side by side
    (None: in their own)."""
    if p.is_contiguous():
        return None
    order = sorted(range(p.dim()), key=lambda k: (-p.stride(k), -p.shape[k]))
    if not p.permute(order).is_contiguous():
        raise ValueError(f"a parameter of strides {p.stride()} does not fill its memory")
    return order


def _on_device(p) -> bool:
    return p.is_cuda


def _capturing(device) -> bool:
    return device.type == "cuda" and torch.cuda.is_current_stream_capturing()


def _refuse_capture(device) -> None:
    """Moments and counts that a graph zeroes would begin anew at each replay."""
    if _capturing(device):
        raise RuntimeError("a parameter's first step cannot be captured: take it before")


_MOST = 1 << 34  # a tensor has fewer elements


def _check_settings(lr, betas, eps, weight_decay, capturable: bool) -> None:
    if isinstance(lr, torch.Tensor):
        if not capturable:
            raise ValueError("lr may be a tensor with capturable=True")
    elif not 0.0 <= lr < float("inf"):
        raise ValueError(f"lr must be finite and not negative, got {lr}")
    if len(betas) != 2 or not all(0.0 <= b < 1.0 for b in betas):
        raise ValueError(f"betas must be two numbers from 0 to below 1, got {betas}")
    if not 0.0 <= eps < float("inf") or not 0.0 <= weight_decay < float("inf"):
        raise ValueError("eps and weight_decay must be finite and not negative")


class AdamW(torch.optim.Optimizer):
    """AdamW (decoupled weight decay) on ROCm devices, all parameters of a
    type in one launch.

    bits=8 keeps both moments in 8 bits, 2 + 1/64 bytes a parameter in place of
    8.  Of a block of 128 elements those whose gradients are below about 2^-17
    of the largest's then take steps that shrink with them, as with a larger
    eps; those near to it take noisy ones, the largest about 1.4 times as long
    as with 32-bit moments.  random rounds bf16 parameters at random (8-bit
    moments always are), so that small updates count.  max_norm clips the
    gradients' norm over all parameters (``last_norm`` is that of the last
    step, on the device).  Nothing waits for the device.

    The random numbers come from `seed`, the step and the parameter's place: a
    process group's ranks, which step with equal gradients, stay equal while
    they have one seed.

    Each parameter counts the steps in which it had a gradient.
    capturable=True counts on the device, so that a captured graph goes on
    counting (and draws new numbers) at each replay; lr may then be a float32
    tensor on the device.  A group's parameters share a count
    (``param_groups[k]["step"]``) while they have gradients in the same steps;
    the others get one of their own, in their state.  That, like a parameter's
    first step, which makes its moments, is done before a capture."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 1e-2, *, bits: int = 32, random: bool = True,
                 seed: int = 0, max_norm: float | None = None, capturable: bool = False):
        if bits not in (8, 32):
            raise ValueError(f"bits must be 8 or 32, got {bits!r}")
        _check_settings(lr, betas, eps, weight_decay, capturable)
        if max_norm is not None and not 0.0 <= max_norm < float("inf"):
            raise ValueError(f"max_norm must be finite and not negative, got {max_norm}")
        super().__init__(params, dict(lr=lr, betas=tuple(betas), eps=eps,
                                      weight_decay=weight_decay))
        self.bits, self.random, self.seed = bits, bool(random), int(seed)
        self.max_norm, self.capturable, self.last_norm = max_norm, bool(capturable), None

    def __getstate__(self):  # torch's holds the groups and states alone
        own = ("bits", "random", "seed", "max_norm", "capturable", "last_norm")
        return {**super().__getstate__(), **{name: getattr(self, name) for name in own}}

    def _new_state(self, p):
        n, device = p.numel(), p.device
        order = _order(p)
        _refuse_capture(device)
        if self.bits == 32:
            state = {"exp_avg": torch.zeros(n, device=device),
                     "exp_avg_sq": torch.zeros(n, device=device)}
        else:
            m, v = Moment8.zeros(n, device, False), Moment8.zeros(n, device, True)
            state = {"exp_avg": m.codes, "exp_avg_exps": m.exps,
                     "exp_avg_sq": v.codes, "exp_avg_sq_exps": v.exps}
        # p's sizes, and the order of its dimensions in which the moments lie
        state["shape"], state["order"] = list(p.shape), order
        if not self.capturable:
            state["step"] = 0
        return state

    def moments(self, p):
        """p's (first, second) moment, flat in the order that p's memory had
        in its first step (``state[p]["order"]`` of its dimensions; None:
        their own): fp32 tensors or Moment8."""
        state = self.state[p]
        if self.bits == 32:
            return state["exp_avg"], state["exp_avg_sq"]
        n = p.numel()
        return (Moment8(state["exp_avg"], state["exp_avg_exps"], n),
                Moment8(state["exp_avg_sq"], state["exp_avg_sq_exps"], n))

    def _check(self):
        """Refuses what a step would, before it has changed anything."""
        for group in self.param_groups:
            _check_settings(group["lr"], group["betas"], group["eps"], group["weight_decay"],
                            self.capturable)
            params = [p for p in group["params"] if p.grad is not None]
            grads = [p.grad for p in params]
            if any(map(_sparse, grads)):
                raise RuntimeError("AdamW takes no sparse gradients")
            devices = dict(zip(map(_device, params), params))
            for device, p in devices.items():
                if not _on_device(p):
                    raise ValueError(f"AdamW takes parameters on a device, one is on {device}")
            for name, tensors in (("a parameter", params), ("a gradient", grads)):
                for dtype in set(map(_dtype_of, tensors)):
                    _dtype(dtype, name)
            if max(map(_numel, params), default=0) >= _MOST:
                raise ValueError("a parameter has 2^34 elements or more")
            if self.capturable and len(devices) > 1:
                raise ValueError("capturable=True takes a group's parameters on one device, got "
                                 f"{sorted(map(str, devices))}")
            if isinstance(group["lr"], torch.Tensor) and devices:
                _scalar(group["lr"], "lr", torch.float32, *devices)

    def _buckets(self):
        """What one call takes: (group, step, place of its first parameter,
        parameters, values and gradients in the moments' order, and those
        values that are copies with where they belong), by group, device,
        types and step (with capturable: its count, None for the group's)."""
        buckets, place = {}, 0
        for k, group in enumerate(self.param_groups):
            first = None  # the count of parameters that begin behind their group
            if self.capturable:
                self._part_counts(group)
            for p in group["params"]:
                place += 1
                if p.grad is None:
                    continue
                g = p.grad
                state = self.state[p]
                if not state:
                    state.update(self._new_state(p))
                    if self.capturable and "step" in group:
                        if first is None:
                            first = torch.zeros(1, dtype=torch.int64, device=p.device)
                        state["step"] = first
                if "order" not in state:  # saved without it
                    state["order"] = _order(p)
                order = state["order"]
                value, g = p.detach(), g.detach()
                if order is not None:
                    value, g = value.permute(order), g.permute(order)
                step = state.get("step")
                key = (k, p.device, p.dtype, g.dtype, id(step) if self.capturable else step)
                if key not in buckets:
                    buckets[key] = (group, step, place, [], [], [], [])
                if not value.is_contiguous():  # p lies in another order since
                    buckets[key][6].append((value, value.contiguous()))
                    value = buckets[key][6][-1][1]
                buckets[key][3].append(p)
                buckets[key][4].append(value)
                buckets[key][5].append(g.contiguous())
        return list(buckets.values())

    def _clip(self, buckets):
        """The gradients' common factor, on the device (None: no clipping)."""
        if self.max_norm is None or not buckets:
            return None
        lists = {}
        for b in buckets:
            for g in b[5]:
                lists.setdefault((g.device, g.dtype), []).append(g)
        if len({device for device, _ in lists}) > 1:
            raise ValueError("max_norm takes parameters on one device")
        if len(lists) == 1:
            self.last_norm, scale = gqs_grad_norm(*lists.values(), max_norm=self.max_norm)
            return scale
        norms = torch.stack([gqs_grad_norm(grads)[0] for grads in lists.values()])
        self.last_norm = norms.double().square().sum().sqrt().float()
        return (self.max_norm / (self.last_norm + 1e-6)).clamp(max=1.0)

    def _part_counts(self, group):
        """Gives those of a count's parameters that have no gradient now a
        count of their own where others have one."""
        params, counts = group["params"], {}
        if all(p.grad is not None for p in params):
            return
        for p in params:
            state = self.state.get(p)
            if state:
                count = state.get("step", group.get("step"))
                counts.setdefault(id(count), (count, [], []))[1 if p.grad is None else 2].append(p)
        for count, still, stepping in counts.values():
            if still and stepping and count is not None:
                if _capturing(count.device):
                    raise RuntimeError("a captured step takes gradients of the parameters that "
                                       "had them before: take one with these before")
                own = count.clone()
                for p in still:
                    self.state[p]["step"] = own

    def _count(self, group, device):
        """The group's number of steps on the device."""
        if group.get("step") is None:
            _refuse_capture(device)
            group["step"] = torch.zeros(1, dtype=torch.int64, device=device)
        return group["step"]

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        self._check()
        buckets = self._buckets()
        if not self.capturable and buckets and _capturing(buckets[0][3][0].device):
            raise RuntimeError("a captured step needs capturable=True: the graph would keep "
                               "the number of this one")
        scale = self._clip(buckets)
        counted = {}
        for group, step, place, params, values, grads, copies in buckets:
            if self.capturable:
                if step is None:
                    step = self._count(group, params[0].device)
                if id(step) not in counted:
                    counted[id(step)] = step.add_(1)
            else:
                step += 1
            m, v = zip(*(self.moments(p) for p in params))
            bf16 = params[0].dtype == torch.bfloat16
            drawn = self.bits == 8 or (self.random and bf16)
            nearest = {"random": False} if drawn and bf16 and not self.random else {}
            gqs_adamw(values, grads, m, v, step=step, lr=group["lr"], betas=group["betas"],
                      eps=group["eps"], weight_decay=group["weight_decay"], scale=scale,
                      seed=_mix_seed(self.seed, place) if drawn else None, **nearest)
            for view, value in copies:
                view.copy_(value)
            if not self.capturable:
                for p in params:
                    self.state[p]["step"] = step
        return loss

    def _check_sizes(self, i, state, p):
        """Whether saved moments are this optimizer's, of a parameter like p."""
        steps = state.get("step")
        if (state and not {"exp_avg", "exp_avg_sq"} <= state.keys()
                or any(v.dim() != 1 for v in state.values() if isinstance(v, torch.Tensor))
                or isinstance(steps, torch.Tensor) and steps.is_floating_point()):
            raise ValueError(f"the state of parameter {i} is another optimizer's")
        if state.get("shape", list(p.shape)) != list(p.shape):
            raise ValueError(f"the state of parameter {i} is of {state['shape']}, its parameter "
                             f"{list(p.shape)}")
        blocks = (p.numel() + 127) // 128
        sizes = {"exp_avg": p.numel()} if self.bits == 32 else {"exp_avg": 128 * blocks,
                                                                "exp_avg_exps": blocks}
        for key, n in sizes.items():
            for name in (key, key.replace("avg", "avg_sq")):
                if name in state and state[name].numel() != n:
                    raise ValueError(f"the state of parameter {i} has {state[name].numel()} "
                                     f"elements of {name}, its parameter takes {n}")

    def load_state_dict(self, state_dict):
        """As torch's, which would cast moments and codes to the parameters'
        types: they come as they were saved, for parameters of the same shapes
        in any memory order.  Steps counted on the host and on the device are
        taken for each other."""
        saved = [i for group in state_dict["param_groups"] for i in group["params"]]
        own = [p for group in self.param_groups for p in group["params"]]
        for i, p in zip(saved, own):
            self._check_sizes(i, state_dict["state"].get(i, {}), p)
        for group in state_dict["param_groups"]:
            states = [state_dict["state"].get(i, {}) for i in group["params"]]
            for state in states:
                codes = state.get("exp_avg")
                if codes is not None and (codes.dtype == torch.float32) != (self.bits == 32):
                    raise ValueError(f"the state has other moments than those of bits={self.bits}")
            counts = {state["step"] for state in states
                      if not isinstance(state.get("step"), (type(None), torch.Tensor))}
            if self.capturable and len(counts) > 1:
                raise ValueError("capturable=True takes one count for a group over from the "
                                 f"host's, the state's are {sorted(counts)}")
        super().load_state_dict(state_dict)
        own = [p for group in self.param_groups for p in group["params"]]
        for i, p in zip(saved, own):
            for key, value in state_dict["state"].get(i, {}).items():
                if isinstance(value, torch.Tensor):
                    value = value.detach().clone().to(p.device)
                elif isinstance(value, list):
                    value = list(value)
                self.state[p][key] = value
        for group in self.param_groups:
            states = [self.state[p] for p in group["params"] if self.state.get(p)]
            common = group.pop("step", None)
            steps = [state.pop("step", common) for state in states]
            steps = [0 if n is None else int(n) for n in steps]
            if not self.capturable:
                for state, n in zip(states, steps):
                    state["step"] = n
            elif steps:
                common = steps[0] if common is None else int(common)
                counts = {n: torch.tensor([n], device=states[0]["exp_avg"].device)
                          for n in {common, *steps}}
                group["step"] = counts[common]
                for state, n in zip(states, steps):
                    if n != common:
                        state["step"] = counts[n]
