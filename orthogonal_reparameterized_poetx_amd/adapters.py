"""Low-rank adapters beside a shared projection (poetx_adapters_forward, poetx_adapters_backward).

Holds the device table of a set of adapters and its workspaces, as torch
tensors on one ROCm device.  Every computation is a call into libpoetx.so.
"""

import torch

from . import _lib as L


class AdapterSet:
    """Adapters of one projection with n inputs and m outputs.

    A, B   lists of matrices [r][n] and [m][r], contiguous, all bfloat16 or all
           float32, kept and read in place; ranks 1..256, they may differ
    scales one factor for each adapter
    dA, dB lists of float32 gradients of the same shapes that backward() writes;
           by default allocated by the first backward() (which then cannot
           be inside a graph capture)

    A batch is cut into segments of consecutive tokens: seg_start (int32,
    one more entry than segments) and seg_adapter (int32, an index into the
    set or -1), both on the device.

    Calls run on the current stream.  Those of one object share its
    workspaces: on several streams at once, use an object for each.  A
    captured graph uses the object's buffers: keep the object as long as it.
    """

    def __init__(self, m, n, A, B, scales, dA=None, dB=None):
        if not A or len(A) != len(B) or len(A) != len(scales):
            raise ValueError("as many A as B and scales, at least one, are needed")
        self.m, self.n = int(m), int(n)
        self.device, self.dtype = A[0].device, A[0].dtype
        if not A[0].is_cuda:
            raise ValueError("adapters are on %s: a ROCm device is needed" % self.device)
        if self.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("adapters are %s (bfloat16 or float32 is needed)" % self.dtype)
        self.A, self.B, self.scales = list(A), list(B), [float(s) for s in scales]
        for i, (a, b) in enumerate(zip(self.A, self.B)):
            r = a.shape[0]
            self._check("A[%d]" % i, a, (r, self.n), self.dtype)
            self._check("B[%d]" % i, b, (self.m, r), self.dtype)
        self.dA, self.dB = self._grads("dA", dA, self.A), self._grads("dB", dB, self.B)
        self._ws, self._need = {}, {}     # workspaces by op; their sizes by (op, tokens, segments)
        self.table = None
        self._make_table()

    def _check(self, name, t, shape, dtype):
        if t.device != self.device or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError("%s must be a contiguous %s tensor of shape %s on %s" % (name, dtype, tuple(shape),
                                                                                     self.device))

    def _grads(self, name, grads, like):
        if grads is None:
            return None
        if len(grads) != len(like):
            raise ValueError("%s has %d entries for %d adapters" % (name, len(grads), len(like)))
        for i, (g, t) in enumerate(zip(grads, like)):
            if g is not None:
                self._check("%s[%d]" % (name, i), g, t.shape, torch.float32)
        return list(grads)

    def _make_table(self):
        none = [None] * len(self.A)
        self._held = [tuple(ts or ()) for ts in (self.A, self.B, self.dA, self.dB)]    # the table has their addresses
        rows = [L.Adapter(L._addr(a), L._addr(b), L._addr(da), L._addr(db), a.shape[0], s)
                for a, b, da, db, s in zip(self.A, self.B, self.dA or none, self.dB or none, self.scales)]
        dt = L.POETX_BF16 if self.dtype == torch.bfloat16 else L.POETX_F32
        host, self.aset = L.adapter_table(rows, self.m, self.n, dt)
        if self.table is None:
            self.table = host.to(self.device)
            self._owned = L.Owned(self.table)
        else:   # in its place: captured graphs hold the address (the pointers of A and B are the same again)
            self.table.copy_(host)
        self.aset.table = self.table.data_ptr()
        torch.cuda.current_stream(self.device).synchronize()

    def _rows(self, name, t, width, N=None):
        """Row stride of an activation matrix."""
        if t.device != self.device or t.dtype != self.dtype or t.dim() != 2 or t.shape[1] != width or \
                (N is not None and t.shape[0] != N) or (width > 1 and t.stride(1) != 1):
            raise ValueError("%s must be a %s matrix [%s][%d] with contiguous rows on %s"
                             % (name, self.dtype, "N" if N is None else N, width, self.device))
        ld = t.stride(0) if t.shape[0] > 1 else width
        if ld < width:
            raise ValueError("rows of %s overlap" % name)
        return ld

    def _segs(self, seg_start, seg_adapter):
        for name, t in (("seg_start", seg_start), ("seg_adapter", seg_adapter)):
            if t.device != self.device or t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
                raise ValueError("%s must be a contiguous int32 vector on %s" % (name, self.device))
        if seg_start.numel() != seg_adapter.numel() + 1:
            raise ValueError("seg_start needs one entry more than seg_adapter")
        return seg_adapter.numel()

    def workspace(self, op, N, nseg, stream=None):
        need = self._need.get((op, N, nseg))
        if need is None:
            if len(self._need) > 4096:
                self._need.clear()
            need = self._need[op, N, nseg] = L.adapters_workspace_bytes(self.aset, N, nseg, op)
        ws = self._ws.get(op)
        if ws is None or ws.numel() < need:
            # the smaller one stays: a captured graph or another stream's queued work may still use it
            # (twice its size at least, so that less is kept than is in use)
            if ws is not None:
                need = max(need, 2 * ws.numel())
            ws = self._ws[op] = self._owned.add(L.make_workspace(need, self.device, stream))
        return ws

    def forward(self, X, Y, seg_start, seg_adapter, stream=None):
        """Y[t] += s B (A X[t]) with each segment's adapter, in place; returns Y."""
        nseg = self._segs(seg_start, seg_adapter)
        N = X.shape[0]
        ldx, ldy = self._rows("X", X, self.n), self._rows("Y", Y, self.m, N)
        handle = self._owned.handle(stream)
        L.poetx_adapters_forward(self.aset, seg_start, seg_adapter, nseg, X, ldx, N, Y, ldy,
                                 self.workspace(L.OP_FORWARD, N, nseg, stream), handle)
        return Y

    def backward(self, X, dY, seg_start, seg_adapter, dX=None, accumulate=False, stream=None):
        """Gradients of sum(dY * forward): adds to dX (if given) and writes,
        or with accumulate adds to, self.dA and self.dB, which it returns."""
        nseg = self._segs(seg_start, seg_adapter)
        N = X.shape[0]
        ldx, lddy = self._rows("X", X, self.n), self._rows("dY", dY, self.m, N)
        lddx = 0 if dX is None else self._rows("dX", dX, self.n, N)
        if self.dA is None or self.dB is None:
            if accumulate:
                raise ValueError("accumulate needs gradients to add to")
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("the first backward makes the gradients: call it before the capture, or give dA and dB")
            self.dA = self.dA or [torch.zeros_like(a, dtype=torch.float32) for a in self.A]
            self.dB = self.dB or [torch.zeros_like(b, dtype=torch.float32) for b in self.B]
            self._make_table()      # waits for the current stream: the gradients are there for any
        self.aset.flags = L.POETX_ACCUMULATE_GRAD if accumulate else 0
        handle = self._owned.handle(stream)
        L.poetx_adapters_backward(self.aset, seg_start, seg_adapter, nseg, X, ldx, dY, lddy, N, dX, lddx,
                                  self.workspace(L.OP_BACKWARD, N, nseg, stream), handle)
        return self.dA, self.dB
