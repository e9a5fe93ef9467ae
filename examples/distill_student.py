"""Distil a small student language model under ZeRO-2, start to end.

N_d data-parallel ranks are emulated on one GPU, as everywhere in this package:
every rank has its own tokens and its own gradient buffer, and one fused step
reduce-scatters, updates and all-gathers.  The model around that step uses the
package's operators for everything but the matrix products:

    ids -> embedding -> [norm -> products -> norm, gate, residual] x blocks
        -> norm -> tied output head -> loss against a teacher's top logits

Weights are read from the replicated bf16 buffer that the step writes, and every
gradient is written to its place in the rank's flat gradient buffer.  The head
is tied to the embedding: its product writes the table's gradient, the
embedding's gradient is added to it.

    python examples/distill_student.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fsdp_sharded_optimizer_gb300 as Z  # noqa: E402

RANKS, VOCAB, DIM, HIDDEN, BLOCKS, TOKENS, TOP = 2, 5003, 256, 512, 2, 1024, 32
TEMPERATURE, CE_WEIGHT, KL_WEIGHT = 2.0, 0.2, 0.8
NORM = dict(kind="rms", eps=1e-5, residual_scale=1.0, branch_scale=0.5)


def shapes():
    """Name -> shape of every parameter, in the order of the flat buffer."""
    out = {"table": (VOCAB, DIM), "first_norm": (DIM,)}
    for b in range(BLOCKS):
        out["up%d" % b] = (HIDDEN, DIM)
        out["down%d" % b] = (DIM, HIDDEN)
        out["post%d" % b] = (DIM,)
        out["gate%d" % b] = (1, DIM)
        out["pre%d" % b] = (DIM,)  # before the next block, or before the head
    return out


def views(flat):
    """The parameters' tensors inside a flat buffer."""
    out, at = {}, 0
    for name, shape in shapes().items():
        n = torch.Size(shape).numel()
        out[name] = flat[at:at + n].view(shape)
        at += n
    return out


class Student:
    """Flat state of the job, and the model's forward and backward pass on it."""

    def __init__(self, seed=0):
        n = sum(torch.Size(s).numel() for s in shapes().values())
        (self.unit,), _ = Z.zero_layout([n], RANKS)
        P, S = self.unit.n_padded, self.unit.shard_len
        gen = torch.Generator(device="cuda").manual_seed(seed)
        start = torch.zeros(P, device="cuda")
        for name, w in views(start).items():
            if w.dim() == 1 or name.startswith("gate"):
                w.fill_(1.0)
            else:
                w.copy_(torch.randn(w.shape, generator=gen, device="cuda") * DIM ** -0.5)
        self.master = start.view(RANKS, S).clone()
        self.m, self.v = torch.zeros_like(self.master), torch.zeros_like(self.master)
        self.params = start.bfloat16()
        self.grads = torch.zeros((RANKS, P), dtype=torch.bfloat16, device="cuda")
        self.w = views(self.params)
        self.scale = DIM ** 0.5
        self.embed_scratch = torch.empty(Z.zero_embed_scratch_bytes(TOKENS, VOCAB, DIM),
                                         dtype=torch.uint8, device="cuda")
        self.norm_scratch = torch.empty(Z.zero_block_norm_scratch_bytes(TOKENS, DIM),
                                        dtype=torch.uint8, device="cuda")

    def forward(self, ids):
        """Logits of the tokens, and what the backward pass needs."""
        w = self.w
        act = dict(dtype=torch.bfloat16, device="cuda")
        x, u = torch.empty((TOKENS, DIM), **act), torch.empty((TOKENS, DIM), **act)
        Z.zero_embed_forward(w["table"], ids, x, scale=self.scale)
        Z.zero_block_norm_forward(x, pre_weight=w["first_norm"], u=u, **NORM)
        kept = []
        for b in range(BLOCKS):
            hidden = torch.relu(u @ w["up%d" % b].t())
            branch = hidden @ w["down%d" % b].t()
            y, u_next = torch.empty_like(x), torch.empty_like(u)
            Z.zero_block_norm_forward(x, branch=branch, gate=w["gate%d" % b],
                                      post_weight=w["post%d" % b], pre_weight=w["pre%d" % b],
                                      y=y, u=u_next, **NORM)
            kept.append((x, u, hidden, branch))
            x, u = y, u_next
        return u @ w["table"].t(), (kept, x, u)

    def backward(self, ids, logits, kept, teacher, labels, grads):
        """Writes the rank's gradients; returns the rows' losses (ce, kl)."""
        w, g = self.w, views(grads)
        kept, x, u = kept
        ce, kl = (torch.empty(TOKENS, device="cuda") for _ in range(2))
        weight = torch.full((TOKENS,), 1.0 / TOKENS, device="cuda")
        Z.zero_distill_forward_backward(logits, *teacher, ce, kl, logits, labels=labels,
                                        row_weight=weight, temperature=TEMPERATURE,
                                        ce_weight=CE_WEIGHT, kl_weight=KL_WEIGHT)
        torch.matmul(logits.t(), u, out=g["table"])
        du, dx = logits @ w["table"], None
        for b in reversed(range(BLOCKS)):
            x_in, u_in, hidden, branch = kept[b]
            dx_in, dbranch = torch.empty_like(x), torch.empty_like(branch)
            Z.zero_block_norm_backward(
                x, self.norm_scratch, dy=dx, du=du, branch=branch, gate=w["gate%d" % b],
                post_weight=w["post%d" % b], pre_weight=w["pre%d" % b], dx=dx_in,
                dbranch=dbranch, dgate=g["gate%d" % b], dpost_weight=g["post%d" % b],
                dpre_weight=g["pre%d" % b], **NORM)
            torch.matmul(dbranch.t(), hidden, out=g["down%d" % b])
            dhidden = (dbranch @ w["down%d" % b]) * (hidden > 0)
            torch.matmul(dhidden.t(), u_in, out=g["up%d" % b])
            du, dx, x = dhidden @ w["up%d" % b], dx_in, x_in
        dembed = torch.empty_like(x)
        Z.zero_block_norm_backward(x, self.norm_scratch, dy=dx, du=du,
                                   pre_weight=w["first_norm"], dx=dembed,
                                   dpre_weight=g["first_norm"], **NORM)
        Z.zero_embed_backward(dembed, ids, g["table"], self.embed_scratch, scale=self.scale,
                              accumulate=True)
        return ce, kl

    def step(self, t, batches, lr=2e-3):
        """One ZeRO-2 step over the ranks' batches; the mean losses of each rank."""
        losses = []
        for rank, (ids, teacher, labels) in enumerate(batches):
            logits, kept = self.forward(ids)
            losses.append(self.backward(ids, logits, kept, teacher, labels, self.grads[rank]))
        Z.zero_step_stage12(2, self.grads, self.master, self.m, self.v, self.params,
                            Z.hparams(lr=lr, step=t), bucket_elems=1 << 20)
        return [(ce.mean(), kl.mean()) for ce, kl in losses]


class Teacher:
    """A fixed distribution of the next token for each token: top logits and ids."""

    def __init__(self, seed=1):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.ids = torch.stack([torch.randperm(VOCAB, generator=gen, device="cuda")[:TOP]
                                for _ in range(64)]).to(torch.int32)
        self.logits = torch.randn((64, TOP), generator=gen, device="cuda").mul_(2.0)
        self.gen = gen

    def batch(self):
        ids = torch.randint(0, VOCAB, (TOKENS,), generator=self.gen, device="cuda")
        row = ids % 64
        labels = self.ids[row, self.logits[row].argmax(1)].long()
        labels[-16:] = -100  # no label at the end: only the teacher's distribution
        return ids, (self.logits[row].contiguous(), self.ids[row].contiguous()), labels


def run(steps=30):
    student, teacher = Student(), Teacher()
    history = []
    for t in range(1, steps + 1):
        losses = student.step(t, [teacher.batch() for _ in range(RANKS)])
        history.append(sum(float(CE_WEIGHT * ce + KL_WEIGHT * kl) for ce, kl in losses) / RANKS)
    return history


if __name__ == "__main__":
    for i, loss in enumerate(run(int(sys.argv[1]) if len(sys.argv) > 1 else 30)):
        print("step %3d  loss %.4f" % (i + 1, loss))
