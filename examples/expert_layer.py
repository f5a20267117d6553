"""A feed-forward layer of experts on the library's operators.

    python examples/expert_layer.py

Training: every token's top_k choices sorted by expert, the rows sent there, the
experts' gated product and down projection, their weighted sum on the residual
stream, and the backward pass of all of it, one HIP graph a step.  Serving: the
same weights in e4m3 with a scale for each block of 128 x 128, rows quantised in
blocks of 128.  PyTorch supplies memory, streams, the router and the optimizer's
update.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import compiler_hlo_amd as H  # noqa: E402


class TrainingStep:
    """y = x + sum_j weight[t, j] down_e(silu(gate_e(x)) * up_e(x)), e =
    expert[t, j], with the gradient of 0.5 |y - target|^2 / tokens in x, in every
    expert's weights and in the choices' weights."""

    def __init__(self, tokens, top_k, experts, hidden, inner, dtype="bf16", seed=0):
        t = torch.bfloat16 if dtype == "bf16" else torch.float16
        g = torch.Generator(device="cuda").manual_seed(seed)
        make = lambda shape, s: torch.randn(shape, generator=g, device="cuda") * s  # noqa: E731
        self.master = {"gate_up": make((experts * 2 * inner, hidden), hidden ** -0.5),
                       "down": make((experts * hidden, inner), inner ** -0.5)}
        self.weight = {k: v.to(t) for k, v in self.master.items()}
        self.x = torch.zeros((tokens, hidden), dtype=t, device="cuda")
        self.target = torch.zeros_like(self.x)
        self.expert = torch.zeros((tokens, top_k), dtype=torch.int32, device="cuda")
        self.share = torch.zeros((tokens, top_k), device="cuda")  # a choice's weight
        w, pairs = self.weight, tokens * top_k
        self.sort = H.ExpertSort(tokens, top_k, experts).bind(self.expert)
        place, _, offsets = self.sort.results
        self.send = H.ExpertDispatch(tokens, top_k, hidden, dtype).bind(self.x, place)
        rows = self.send.results
        self.up = H.GatedFeedForward(pairs, inner, hidden, dtype, save=True, experts=experts).bind(rows, w["gate_up"], offsets)
        a, z = self.up.results
        self.down = H.Matmul(pairs, hidden, inner, dtype, experts=experts).bind(a, w["down"], offsets)
        self.back = H.ExpertCombine(tokens, top_k, hidden, dtype, residual=True).bind(self.down.results, place, self.share, self.x)
        self.y = self.back.results
        self.dy = torch.zeros_like(self.x)
        self.dback = H.ExpertCombineGrad(tokens, top_k, hidden, dtype).bind(self.dy, self.down.results, place, self.share)
        drows, self.grad_share = self.dback.results
        self.ddown = H.MatmulGrad(pairs, hidden, inner, dtype, experts=experts).bind(drows, a, w["down"], offsets)
        da, self.grad_down = self.ddown.results
        self.dup = H.GatedFeedForwardGrad(pairs, inner, hidden, dtype, experts=experts).bind(da, rows, w["gate_up"], z, offsets)
        dsent, self.grad_gate_up = self.dup.results
        # the dispatch's gradient, and the residual's beside it
        self.dsend = H.ExpertCombine(tokens, top_k, hidden, dtype, weighted=False, residual=True).bind(dsent, place, self.dy)
        self.dx = self.dsend.results
        self.graph = None

    def route(self, scores):
        """The choices of a router's scores [tokens, experts]."""
        value, chosen = scores.topk(self.expert.shape[1], 1)
        self.expert.copy_(chosen)
        self.share.copy_(torch.softmax(value, 1))

    def forward(self):
        for launch in (self.sort, self.send, self.up, self.down, self.back):
            launch()

    def backward(self):
        torch.sub(self.y, self.target, out=self.dy)
        self.dy.mul_(1.0 / self.y.shape[0])
        for launch in (self.dback, self.ddown, self.dup, self.dsend):
            launch()

    def loss(self):
        return 0.5 * float((self.y.float() - self.target.float()).square().sum()) / self.y.shape[0]

    def capture(self):
        """Forward and backward as one graph; replays read the choices, x, target
        and the weights as they are then."""
        self.forward(), self.backward()
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.forward(), self.backward()

    def step(self, lr):
        if self.graph is None:
            self.capture()
        self.graph.replay()
        for name, grad in (("gate_up", self.grad_gate_up), ("down", self.grad_down)):
            self.master[name].sub_(grad.float(), alpha=lr)
            self.weight[name].copy_(self.master[name])


class Served:
    """The layer in e4m3 with block scales: weights laid out once, an expert's
    blocks after another's; rows quantised before each product."""

    def __init__(self, master, experts):
        self.experts = experts
        self.hidden, self.inner = master["down"].shape[0] // experts, master["down"].shape[1]
        # gate and up have blocks of their own: 2 * experts parts
        self.gate_up, self.gate_up_scale = self.quantise(master["gate_up"], 2 * experts)
        self.down, self.down_scale = self.quantise(master["down"], experts)
        self.ops = {}

    @staticmethod
    def quantise(w, parts):
        rows, cols = w.shape[0] // parts, w.shape[1]
        high, wide = -(-rows // 128), -(-cols // 128)
        padded = torch.nn.functional.pad(w.reshape(parts, rows, cols), (0, wide * 128 - cols, 0, high * 128 - rows))
        blocks = padded.reshape(parts, high, 128, wide, 128)
        scale = blocks.abs().amax((2, 4)) / 448.0
        q = (blocks / torch.where(scale > 0, scale, 1.0)[:, :, None, :, None]).clamp(-448.0, 448.0)
        q = q.reshape(parts, high * 128, wide * 128)[:, :rows, :cols].reshape(parts * rows, cols)
        return q.to(torch.float8_e4m3fn).contiguous(), scale.reshape(parts * high, wide).contiguous()

    def __call__(self, x, expert, share):
        """y for any number of tokens."""
        tokens, top_k = expert.shape
        if (tokens, top_k) not in self.ops:  # handles cost microseconds and no compile
            pairs, f8 = tokens * top_k, dict(dtype="f8e4m3", scales="blocks", experts=self.experts)
            self.ops[tokens, top_k] = (H.ExpertSort(tokens, top_k, self.experts), H.BlockQuantize(tokens, self.hidden),
                                       H.ExpertDispatch(tokens, top_k, self.hidden, "f8e4m3", scales="blocks"),
                                       H.GatedFeedForward(pairs, self.inner, self.hidden, **f8),
                                       H.BlockQuantize(pairs, self.inner), H.Matmul(pairs, self.hidden, self.inner, **f8),
                                       H.ExpertCombine(tokens, top_k, self.hidden, residual=True))
        sort, quantise, send, up, again, down, back = self.ops[tokens, top_k]
        place, _, offsets = sort(expert)
        q, scale = quantise(x)
        rows, rows_scale = send(q, place, scale)
        h, h_scale = again(up(rows, self.gate_up, rows_scale, self.gate_up_scale, offsets))
        return back(down(h, self.down, h_scale, self.down_scale, offsets), place, share, x)


def main():
    tokens, top_k, experts, hidden, inner = 1000, 2, 8, 512, 704
    layer = TrainingStep(tokens, top_k, experts, hidden, inner)
    g = torch.Generator(device="cuda").manual_seed(1)
    layer.x.copy_(torch.randn(layer.x.shape, generator=g, device="cuda"))
    layer.target.copy_(layer.x.roll(1, 1))
    router = torch.randn((hidden, experts), generator=g, device="cuda") * hidden ** -0.5
    layer.route(layer.x.float() @ router)
    for i in range(21):
        layer.step(lr=0.02)
        if i % 5 == 0:
            print("step %2d  loss %.3f" % (i, layer.loss()), flush=True)
    served = Served(layer.master, experts)
    for n in (1, 7, 1000):
        y = served(layer.x[:n].contiguous(), layer.expert[:n].contiguous(), layer.share[:n].contiguous())
        print("served %4d tokens, loss %.3f" % (n, 0.5 * float((y.float() - layer.target[:n].float()).square().sum()) / n))


if __name__ == "__main__":
    main()
