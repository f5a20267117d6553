"""A transformer's feed-forward layer on the library's operators.

    python examples/feed_forward.py

Training: norm of the residual stream, gated product, down projection,
dropout and the residual's addition, and their backward pass, one HIP graph a
step.  Serving: the same weights in 8 bits, rows quantised by the norm, for a
prompt and for single tokens.  PyTorch supplies memory, streams and the
optimizer's update.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import compiler_hlo_amd as H  # noqa: E402


class TrainingStep:
    """y = x + dropout(down(silu(gate(h)) * up(h))), h = norm(x), with the
    gradient of 0.5 |y - target|^2 / rows in every weight and in x."""

    def __init__(self, rows, hidden, inner, dtype="bf16", p=0.1, seed=0):
        t = torch.bfloat16 if dtype == "bf16" else torch.float16
        g = torch.Generator(device="cuda").manual_seed(seed)
        make = lambda shape, s: torch.randn(shape, generator=g, device="cuda") * s  # noqa: E731
        # the weights in f32 for the update, and what the products read
        self.master = {"norm": torch.ones(hidden, device="cuda"),
                       "gate_up": make((2 * inner, hidden), hidden ** -0.5),
                       "down": make((hidden, inner), inner ** -0.5)}
        self.weight = {k: v.to(t) for k, v in self.master.items()}
        self.x = torch.zeros((rows, hidden), dtype=t, device="cuda")
        self.target = torch.zeros_like(self.x)
        self.state = torch.tensor([seed, 0], dtype=torch.int64, device="cuda")
        self.counters = -(-rows * hidden // 8)  # that a step's mask takes
        w = self.weight
        self.norm = H.RmsNorm(rows, hidden, dtype).bind(self.x, w["norm"])
        h, self.rstd = self.norm.results
        self.gated = H.GatedFeedForward(rows, inner, hidden, dtype, save=True).bind(h, w["gate_up"])
        a, z = self.gated.results
        self.down = H.Matmul(rows, hidden, inner, dtype).bind(a, w["down"])
        self.drop = H.Dropout(rows, hidden, dtype, p=p, residual=True).bind(self.down.results, self.state, self.x)
        self.y = self.drop.results
        self.dy = torch.zeros_like(self.x)
        self.ddrop = H.Dropout(rows, hidden, dtype, p=p).bind(self.dy, self.state)
        self.ddown = H.MatmulGrad(rows, hidden, inner, dtype).bind(self.ddrop.results, a, w["down"])
        da, self.grad_down = self.ddown.results
        self.dgated = H.GatedFeedForwardGrad(rows, inner, hidden, dtype).bind(da, h, w["gate_up"], z)
        dh, self.grad_gate_up = self.dgated.results
        # the residual's gradient comes in as the stream's
        self.dnorm = H.RmsNormGrad(rows, hidden, dtype, stream_grad=True).bind(dh, self.x, w["norm"], self.rstd, self.dy)
        self.dx, self.grad_norm = self.dnorm.results
        self.graph = None

    def forward(self):
        for launch in (self.norm, self.gated, self.down, self.drop):
            launch()

    def backward(self):
        torch.sub(self.y, self.target, out=self.dy)
        self.dy.mul_(1.0 / self.y.shape[0])
        for launch in (self.ddrop, self.ddown, self.dgated, self.dnorm):
            launch()

    def loss(self):
        return 0.5 * float((self.y.float() - self.target.float()).square().sum()) / self.y.shape[0]

    def capture(self):
        """Forward and backward as one graph; replays read x, target, state and
        the weights as they are then."""
        self.forward(), self.backward()
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.forward(), self.backward()

    def step(self, lr):
        if self.graph is None:
            self.capture()
        self.graph.replay()
        self.state[1] += self.counters
        for name, grad in (("norm", self.grad_norm), ("gate_up", self.grad_gate_up), ("down", self.grad_down)):
            self.master[name].sub_(grad.float(), alpha=lr)
            self.weight[name].copy_(self.master[name])


class Served:
    """The layer in 8 bits: weights with a scale a channel, laid out once; rows
    quantised by the norm and, between the products, by a norm with weights of
    one, whose rstd the product's row scales take back."""

    def __init__(self, master, kind="f8e4m3"):
        self.kind, self.top = kind, {"f8e4m3": 448.0, "s8": 127.0}[kind]
        self.norm = master["norm"].to(torch.bfloat16)
        self.gate_up, self.gate_up_scale = self.quantise(master["gate_up"])
        self.down, self.down_scale = self.quantise(master["down"])
        self.ones = torch.ones(self.down.shape[1], dtype=torch.bfloat16, device=self.down.device)
        self.ops = {}

    def quantise(self, w):
        scale = w.abs().amax(1) / self.top
        q = (w / torch.where(scale > 0, scale, 1.0)[:, None]).clamp(-self.top, self.top)
        return (q.round().to(torch.int8) if self.kind == "s8" else q.to(torch.float8_e4m3fn)), scale

    def __call__(self, x, residual):
        """(y, the stream before the layer) for any number of rows."""
        rows, hidden = x.shape
        inner = self.down.shape[1]
        if rows not in self.ops:  # handles cost microseconds and no compile
            self.ops[rows] = (H.RmsNorm(rows, hidden, "bf16", residual=True, out_dtype=self.kind),
                              H.GatedFeedForward(rows, inner, hidden, self.kind, out_dtype="bf16"),
                              H.RmsNorm(rows, inner, "bf16", out_dtype=self.kind),
                              H.Matmul(rows, hidden, inner, self.kind, residual=True))
        norm, gated, unit, down = self.ops[rows]
        q, scale, stream, _ = norm(x, self.norm, residual)
        h = gated(q, self.gate_up, scale, self.gate_up_scale)
        # q scale is h rstd, so the rows themselves are q (scale / rstd)
        q, scale, rstd = unit(h, self.ones)
        return down(q, self.down, scale / rstd, self.down_scale, stream), stream


def main():
    rows, hidden, inner = 1000, 1024, 2816
    layer = TrainingStep(rows, hidden, inner)
    g = torch.Generator(device="cuda").manual_seed(1)
    layer.x.copy_(torch.randn(layer.x.shape, generator=g, device="cuda"))
    layer.target.copy_(layer.x.roll(1, 1))
    for i in range(21):
        layer.step(lr=0.02)
        if i % 5 == 0:
            print("step %2d  loss %.3f" % (i, layer.loss()), flush=True)
    served = Served(layer.master)
    for rows in (1, 7, 1000):
        x = layer.x[:rows].contiguous()
        y, _ = served(x, torch.zeros_like(x))
        print("served %4d rows, loss %.3f" % (rows, 0.5 * float((y.float() - layer.target[:rows].float()).square().sum()) / rows))


if __name__ == "__main__":
    main()
