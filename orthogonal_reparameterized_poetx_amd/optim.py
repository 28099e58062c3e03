"""Optimizer steps over many tensors at once (poetx_grad_norm, poetx_adamw_step).

Holds the device table that describes a set of tensors and the flat moment
arrays, as torch tensors on one ROCm device.  Every computation is a call into
libpoetx.so.
"""

import torch

from . import _lib as L

BLOCK = 256   # values that share an exponent byte of an 8-bit state


def _dtype(t, what):
    if t.dtype == torch.float32:
        return L.POETX_F32
    if t.dtype == torch.bfloat16:
        return L.POETX_BF16
    raise ValueError("%s: dtype %s (float32 or bfloat16 is needed)" % (what, t.dtype))


def _flat(t, what, device):
    if not t.is_cuda or t.device != device:
        raise ValueError("%s is on %s, not on %s" % (what, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s is not contiguous" % what)
    return t


def _table(params, grads, copies, lr_mul, decay):
    """(device table, ParamSet, device) of lists of tensors; params may be None (norm only)."""
    if not grads:
        raise ValueError("no tensors")
    device = grads[0].device
    if not grads[0].is_cuda:
        raise ValueError("gradient 0 is on %s: a ROCm device is needed" % device)
    for name, x in (("params", params), ("copies", copies), ("lr_mul", lr_mul), ("weight_decay", decay)):
        if x is not None and len(x) != len(grads):
            raise ValueError("%s has %d entries for %d gradients" % (name, len(x), len(grads)))
    rows = []
    for i, g in enumerate(grads):
        _flat(g, "gradient %d" % i, device)
        p = None if params is None else _flat(params[i], "parameter %d" % i, device)
        c = None if copies is None else copies[i]
        if p is not None and p.numel() != g.numel():
            raise ValueError("parameter %d has %d values, its gradient %d" % (i, p.numel(), g.numel()))
        if c is not None:
            _flat(c, "copy %d" % i, device)
            if c.dtype != torch.bfloat16 or c.numel() != g.numel():
                raise ValueError("copy %d must be bfloat16 with %d values" % (i, g.numel()))
        rows.append(L.Param(L._addr(p), L._addr(g), L._addr(c), g.numel(),
                            1.0 if lr_mul is None else float(lr_mul[i]), 0.0 if decay is None else float(decay[i]),
                            L.POETX_F32 if p is None else _dtype(p, "parameter %d" % i), _dtype(g, "gradient %d" % i)))
    host, pset = L.param_table(rows)
    table = host.to(device)
    pset.table = table.data_ptr()
    return table, pset, device


class GradNorm:
    """norm, coef = GradNorm(grads)(max_norm): the 2-norm of all gradients
    together and min(1, max_norm / (norm + 1e-6)), 0-d fp32 tensors on the
    device that the next call overwrites (coef is NaN where the norm is not
    finite).  Calls on one object must follow each other on one stream.  The
    gradients are read in place by address: other tensors need another object."""

    def __init__(self, grads, _shared=None):
        self.grads = list(grads)
        self._held = tuple(self.grads)      # the table has their addresses
        self.table, self.pset, self.device = _shared or _table(None, self.grads, None, None, None)
        self.out = torch.zeros(2, dtype=torch.float32, device=self.device)
        self.ws = L.make_workspace(L.grad_norm_workspace_bytes(self.pset), self.device)
        self._views = self.out[0], self.out[1]
        self._owned = L.Owned(self.table, self.out, self.ws)
        torch.cuda.current_stream(self.device).synchronize()

    def __call__(self, max_norm=float("inf"), stream=None):
        L.poetx_grad_norm(self.pset, max_norm, self.out, self.ws, self._owned.handle(stream))
        return self._views


class AdamW:
    """AdamW over a list of tensors (fp32 or bf16), one launch a step.

    params, grads  lists of contiguous tensors, kept and read in place: a
                   gradient is written into its tensor before every step
                   (the device table has their addresses: other tensors, such
                   as gradients allocated anew, need another object)
    lr_mul, weight_decay  one value for each tensor (1 and 0 by default)
    copies         for fp32 tensors: bf16 tensors that receive the updated
                   values (entries may be None)
    state_bits     32: fp32 moments; 8: codes with an exponent byte for each 256
                   values, 2 bytes a value in all (include/poetx.h has the format)
    state          moments to start from: a dict of the arrays of state()
    step           steps already taken
    """

    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, lr_mul=None, weight_decay=None,
                 copies=None, state_bits=32, state=None, step=0):
        if state_bits not in (8, 32):
            raise ValueError("state_bits is 8 or 32")
        self.params, self.grads = list(params), list(grads)
        self.copies = None if copies is None else list(copies)
        self._held = tuple(self.params), tuple(self.grads), tuple(self.copies or ())   # the table has their addresses
        self.table, self.pset, self.device = _table(self.params, self.grads, self.copies, lr_mul, weight_decay)
        self.state_bits, self._calls = state_bits, int(step)
        self.hyper = L.AdamwHyper(float(lr), float(betas[0]), float(betas[1]), float(eps))
        nb = self.pset.blocks
        sizes = dict(m=nb * BLOCK, v=nb * BLOCK)
        if state_bits == 8:
            sizes.update(m_exp=nb, v_exp=nb)
        dt = torch.uint8 if state_bits == 8 else torch.float32
        self._state = {}
        self._skipped = torch.zeros(2, dtype=torch.int32, device=self.device)
        for k, n in sizes.items():
            t = torch.zeros(n, dtype=dt, device=self.device) if state is None else state[k]
            if t.dtype != dt or t.numel() != n:
                raise ValueError("state %s must be %s with %d values" % (k, dt, n))
            self._state[k] = _flat(t, "state " + k, self.device)
        self._cstate = L.AdamwState(L._addr(self._state["m"]), L._addr(self._state["v"]),
                                    L._addr(self._state.get("m_exp")), L._addr(self._state.get("v_exp")),
                                    L.POETX_STATE_8BIT if state_bits == 8 else L.POETX_STATE_F32, 0,
                                    self._skipped.data_ptr())
        self._owned = L.Owned(self.table, self._skipped, *self._state.values())
        # here, not at its first call: that may be inside a graph capture (waits for the current stream)
        self._norm = GradNorm(self.grads, (self.table, self.pset, self.device))

    @property
    def lr(self):
        return self.hyper.lr

    @lr.setter
    def lr(self, value):
        self.hyper.lr = float(value)

    @property
    def steps(self):
        """Steps taken: those whose coefficient was not finite are not among them (waits for the device)."""
        torch.cuda.synchronize(self.device)
        return self._calls - int(self._skipped[(self._calls + 1) % 2])

    @steps.setter
    def steps(self, value):
        torch.cuda.synchronize(self.device)
        self._calls = int(value)
        self._skipped.zero_()
        torch.cuda.synchronize(self.device)

    def state(self):
        """The state arrays themselves (save them with self.steps)."""
        return dict(self._state)

    def grad_norm(self, max_norm=float("inf"), stream=None):
        """(norm, coef) of these gradients, as GradNorm."""
        return self._norm(max_norm, stream)

    def step(self, coef=None, stream=None):
        """One step; coef: fp32 tensor of one value on the device that every
        gradient is multiplied by (where it is not finite, it is as if there
        had been no step).  The step's number and learning rate are fixed when
        a graph captures it: every replay repeats them."""
        if coef is not None and (coef.numel() != 1 or coef.dtype != torch.float32 or coef.device != self.device):
            raise ValueError("coef must be one float32 value on %s" % self.device)
        L.poetx_adamw_step(self.pset, self._cstate, self.hyper, self._calls + 1, coef, self._owned.handle(stream))
        self._calls += 1

    def moments(self, out=None, stream=None):
        """(m, v) of the whole set, 256 values a block: the fp32 arrays
        themselves, or what the 8-bit codes stand for (bf16, exact), in `out`
        if that is given: bf16 tensors of as many values (None: not wanted)."""
        if self.state_bits == 32:
            if out is not None:
                raise ValueError("out goes with an 8-bit state: 32-bit moments are returned as they are held")
            return self._state["m"], self._state["v"]
        n = self.pset.blocks * BLOCK
        if out is None:
            m, v = [torch.empty(n, dtype=torch.bfloat16, device=self.device) for _ in range(2)]
            if stream is not None:
                L.lend((m, v), stream)
        else:
            if len(out) != 2:
                raise ValueError("out is a pair, for m and v")
            for name, t in zip("mv", out):
                if t is not None and (_flat(t, "output of " + name, self.device).dtype != torch.bfloat16 or
                                      t.numel() != n):
                    raise ValueError("output of %s must be bfloat16 with %d values" % (name, n))
            m, v = out
        L.poetx_adamw_moments(self.pset, self._cstate, m, v, self._owned.handle(stream))
        return m, v
