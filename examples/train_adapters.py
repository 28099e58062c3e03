"""Trains low-rank adapters of several tasks together with a POET-X layer's
generators, then serves single tokens of many requests.

One step: the shared projection's forward and the adapters' beside it, the
backward of both, the norm of all gradients together, and one AdamW step over
every tensor (generators in fp32; adapters as fp32 master values whose bf16
copies the products read), moments in 8 bits.  Data is synthetic: each task
has a teacher adapter on the same frozen weight.

    python examples/train_adapters.py [--steps 200] [--width 1024] [--tasks 4] [--rank 16] [--state-bits 8]
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import orthogonal_reparameterized_poetx_amd as P  # noqa: E402


def segments(lens, which, device):
    """seg_start, seg_adapter of consecutive segments."""
    start = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(device)
    return start, torch.tensor(which, dtype=torch.int32, device=device)


class Model:
    def __init__(self, width, tasks, rank, state_bits, device="cuda:0", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, sigma):
            return torch.randn(*shape, generator=gen, device=device) * sigma
        self.device, self.width, self.tasks, self.gen = device, width, tasks, gen
        self.layer = P.PoetxLayer(width, width, 64, "bf16", device, perm_seed=seed)
        self.layer.pack(normal(width, width, sigma=width ** -0.5).to(torch.bfloat16))
        # fp32 master values; the adapters the products read are their bf16 copies
        A = [normal(rank, width, sigma=width ** -0.5) for _ in range(tasks)]
        B = [torch.zeros(width, rank, device=device) for _ in range(tasks)]
        master = A + B
        half = [t.to(torch.bfloat16) for t in master]
        dA, dB = [torch.zeros_like(t) for t in A], [torch.zeros_like(t) for t in B]
        self.adapters = P.AdapterSet(width, width, half[:tasks], half[tasks:], [2.0] * tasks, dA=dA, dB=dB)
        self.dth = torch.zeros_like(self.layer.thR), torch.zeros_like(self.layer.thP)
        self.opt = P.AdamW([self.layer.thR, self.layer.thP] + master, list(self.dth) + dA + dB,
                           lr_mul=[0.1, 0.1] + [1.0] * (2 * tasks), weight_decay=[0.0, 0.0] + [0.01] * (2 * tasks),
                           copies=[None, None] + half, state_bits=state_bits, lr=3e-3)
        # the teachers' adapters, on the untrained layer
        self.teacher = P.AdapterSet(width, width, [normal(4, width, sigma=width ** -0.5).to(torch.bfloat16)
                                                   for _ in range(tasks)],
                                    [normal(width, 4, sigma=0.5).to(torch.bfloat16) for _ in range(tasks)],
                                    [1.0] * tasks)
        self.frozen = P.PoetxLayer(width, width, 64, "bf16", device, perm_seed=seed)
        self.frozen.W0p.copy_(self.layer.W0p)
        self.frozen.sigma.copy_(self.layer.sigma)
        self.frozen.tau.copy_(self.layer.tau)

    def forward(self, X, seg):
        """The shared projection, and each segment's adapter beside it."""
        return self.adapters.forward(X, self.layer.forward(X), *seg)

    def step(self, lens, which):
        seg = segments(lens, which, self.device)
        N = sum(lens)
        X = torch.randn(N, self.width, generator=self.gen, device=self.device).to(torch.bfloat16)
        want = self.teacher.forward(X, self.frozen.forward(X), *seg)
        diff = self.forward(X, seg).float() - want.float()
        dY = (diff / N).to(torch.bfloat16)
        dX, _, _ = self.layer.backward(X, dY, dthR=self.dth[0], dthP=self.dth[1])
        self.adapters.backward(X, dY, *seg, dX=dX)      # dX: for a layer below
        norm, coef = self.opt.grad_norm(max_norm=1.0)
        self.opt.step(coef=coef)
        return diff.square().mean(), norm


def train(steps=200, width=1024, tasks=4, rank=16, state_bits=8, log=print):
    """(model, losses): ragged batches, every task in each."""
    model = Model(width, tasks, rank, state_bits)
    lens = [64 * (1 + i % 3) - i % 2 for i in range(2 * tasks)]
    losses = []
    for i in range(steps):
        loss, norm = model.step(lens, [k % tasks for k in range(2 * tasks)])
        losses.append(float(loss))
        if i % 20 == 0 or i == steps - 1:
            log("step %4d  loss %.4f  gradient norm %.4f" % (i, losses[-1], float(norm)))
    return model, losses


def serve(model, requests=48):
    """(outputs of single tokens of many requests in one call, the same tokens of each task as one segment)."""
    X = torch.randn(requests, model.width, device=model.device).to(torch.bfloat16)
    task = [i * model.tasks // requests for i in range(requests)]
    one = model.forward(X, segments([1] * requests, task, model.device))
    runs = [task.count(t) for t in range(model.tasks)]
    whole = model.forward(X, segments(runs, list(range(model.tasks)), model.device))
    return one, whole


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--tasks", type=int, default=4)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=8)
    args = ap.parse_args()
    m, loss = train(args.steps, args.width, args.tasks, args.rank, args.state_bits)
    one, whole = serve(m)
    print("loss %.4f -> %.4f; serving single tokens against whole segments: largest difference %.3g"
          % (loss[0], loss[-1], float((one.float() - whole.float()).abs().max())))
