"""A one-layer mixture-of-experts language model, trained by distillation and
then answering token by token.

    x      = sqrt(H) * table[ids]                         MoKEmbedding
    h      = x + moe(x)                                   MoKRouter, MoKLayer
    logits = h Whead                                      the dense tensor-core GEMM
    loss   = KL(teacher's top logits || student)          DistillLoss, loss and gradient in one call

The teacher is a table: for each token the ids and logits of its most likely
successors.  The student answers through MoKDecoder: the router and the layer
for the few tokens of a serving step in one launch, on the same weights.

    python examples/small_model.py [steps]
"""

import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from mixture_experts_layer_side_gb300 import _lib
from mixture_experts_layer_side_gb300.decode import MoKDecoder
from mixture_experts_layer_side_gb300.distill import DistillLoss
from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
from mixture_experts_layer_side_gb300.inputs import Shape
from mixture_experts_layer_side_gb300.layer import MoKLayer, MoKRouter

VOCAB, TOP, SHAPE = 512, 8, Shape(T=1024, H=256, I=128, E=8, k=2)
LR = {"table": 2.0, "Wr": 0.1, "W1": 2.0, "W3": 2.0, "W2": 2.0, "head": 2.0}


class SmallModel:
    def __init__(self, seed=0):
        s, g = SHAPE, torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape, std):
            return std * torch.randn(shape, generator=g, device="cuda")

        # f32 weights and the bf16 copies that the kernels read
        self.master = {"table": randn(VOCAB, s.H, std=1 / math.sqrt(s.H)), "Wr": randn(s.H, s.E, std=0.05),
                       "W1": randn(s.E, s.H, s.I, std=0.06), "W3": randn(s.E, s.H, s.I, std=0.06),
                       "W2": randn(s.E, s.I, s.H, std=0.06), "head": randn(s.H, VOCAB, std=0.02)}
        self.w = {n: v.bfloat16() for n, v in self.master.items()}
        self.embedding = MoKEmbedding(VOCAB, s.H, s.T)
        self.router, self.layer = MoKRouter(s), MoKLayer(s)
        self.loss = DistillLoss(s.T, VOCAB, TOP)
        self.scratch = torch.zeros(256, dtype=torch.uint8, device="cuda")
        self.scale = math.sqrt(s.H)

    def gemm(self, A, a_mn, B, b_mn, rows, cols):
        C = torch.empty((rows, cols), device="cuda")
        _lib.mok_gemm_bf16(A, a_mn, B, b_mn, C, self.scratch)
        return C

    def forward(self, ids):
        w = self.w
        x = self.embedding.forward(w["table"], ids, scale=self.scale)
        idx, scores = self.router.forward(x, w["Wr"])
        self.layer.build_schedule(idx)
        h = x + self.layer.forward(x, scores, w["W1"], w["W3"], w["W2"])
        return x, idx, scores, h, self.gemm(h, 0, w["head"], 1, SHAPE.T, VOCAB)

    def train_step(self, ids, top_ids, top_logits):
        """One step of gradient descent on the mean loss; returns it (a device tensor)."""
        s, w = SHAPE, self.w
        x, idx, scores, h, logits = self.forward(ids)
        weight = torch.full((s.T,), 1.0 / s.T, device="cuda")
        loss, dz = self.loss.forward_backward(logits, top_ids, top_logits, weight, out=logits)
        dz = dz.bfloat16()
        grads = {"head": self.gemm(h, 1, dz, 1, s.H, VOCAB)}
        dh = self.gemm(dz, 0, w["head"], 0, s.T, s.H).bfloat16()
        g = self.layer.backward(x, scores, w["W1"], w["W3"], w["W2"], dh)
        grads.update(W1=g["dW1"], W3=g["dW3"], W2=g["dW2"])
        grads["Wr"], dx = self.router.backward(x, w["Wr"], idx, scores, g["ds"])
        grads["table"] = self.embedding.backward(dh + g["dX"] + dx, ids, scale=self.scale)
        for n, v in self.master.items():
            v -= LR[n] * grads[n].float()
            self.w[n].copy_(v)
        return loss.mean()

    def check(self):
        for part in (self.embedding, self.router, self.layer, self.loss):
            part.check()


class Answers:
    """The model for up to ``batch`` sequences, one token each a step."""

    def __init__(self, model, batch):
        s = SHAPE
        self.model, self.batch = model, batch
        self.decoder = MoKDecoder(Shape(batch, s.H, s.I, s.E, s.k))
        self.rows = torch.zeros((128, s.H), dtype=torch.bfloat16, device="cuda")  # the GEMM's rows come in 128s

    def logits(self, ids):
        m, w, n = self.model, self.model.w, ids.numel()
        x = m.embedding.forward(w["table"], ids, scale=m.scale)
        out, _, _ = self.decoder.layer(x, w["Wr"], w["W1"], w["W3"], w["W2"])
        self.rows[:n] = x + out
        return m.gemm(self.rows, 0, w["head"], 1, 128, VOCAB)[:n]

    def generate(self, ids, steps):
        """Greedy continuations: int32 [batch, steps]."""
        got = []
        for _ in range(steps):
            ids = self.logits(ids).argmax(1).int()
            got.append(ids)
        return torch.stack(got, 1)


def teacher(seed=1):
    """For each token TOP distinct successors and their logits, the first the most likely."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(VOCAB, generator=g)[:TOP] for _ in range(VOCAB)])
    logits = torch.sort(2.0 * torch.randn((VOCAB, TOP), generator=g), dim=1, descending=True)[0]
    logits[:, 0] += 1.0
    return ids.int().cuda(), logits.cuda()


def train(steps, seed=0):
    model = SmallModel(seed)
    top_ids, top_logits = teacher()
    g = torch.Generator().manual_seed(seed)
    losses = []
    for _ in range(steps):
        ids = torch.randint(0, VOCAB, (SHAPE.T,), generator=g).int().cuda()
        losses.append(model.train_step(ids, top_ids[ids.long()].contiguous(), top_logits[ids.long()].contiguous()))
    model.check()
    return model, top_ids, [float(v) for v in losses]


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 200
    model, top_ids, losses = train(steps)
    print("loss: first %.3f, last %.3f" % (losses[0], losses[-1]))
    answers = Answers(model, 16)
    start = torch.arange(16, device="cuda").int()
    out = answers.generate(start, 12)
    answers.decoder.check()
    before = torch.cat([start[:, None], out[:, :-1]], 1).long()
    print("answers that are the teacher's first choice: %.0f%%" % (100 * (out == top_ids[before, 0]).float().mean()))


if __name__ == "__main__":
    main()
