"""Train a small stack of MLP blocks with the block norm and AdamW.

Every block is  y = x + gain * rms(MLP(n)),  n' = rms(y):  the tensor-parallel
MLP between a pre-norm and a post-norm with a learned gain per channel.  The
norm that ends one block and begins the next, the residual add and the gain are
one kernel forward and one pass backward (TPBlockNorm); all parameters take one
clipped AdamW step (TPAdamW), with states in 8 or 32 bits.  A whole step is
captured into a CUDA graph: the step count, the clip factor and the check that
the gradients are finite stay on the device.

    python examples/train_blocks.py [--blocks 3] [--steps 60] [--state-bits 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tensor_transformer_mlp_shard_gb300 as tp  # noqa: E402


class BlockStack:
    """Blocks, their buffers and one training step towards a target."""

    def __init__(self, blocks=3, S=128, B=2, H=256, F=1024, T=2, state_bits=8, lr=2e-3, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        bf, f32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.float32, device="cuda")
        M, Fs, self.lr = S * B, F // T, lr

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()

        self.mlp = tp.TPMLP(S=S, B=B, H=H, F=F, T=T, act="gelu_tanh", has_bias=True)
        self.first = tp.TPBlockNorm(S, B, H, pre="rms", block=False)
        self.join = tp.TPBlockNorm(S, B, H, post="rms", pre="rms", gate="channel")
        self.x = normal(M, H)
        self.target = normal(M, H)
        self.norm_w = [torch.ones(H, **bf) for _ in range(blocks + 1)]  # the pre-norms, the last one the output's
        self.layers, params, grads, decay = [], [], [], []

        def own(p, wd=0.0):
            g = torch.zeros(p.shape, **f32)
            params.append(p)
            grads.append(g)
            decay.append(wd)
            return g

        self.d_norm_w = [own(w) for w in self.norm_w]
        for _ in range(blocks):
            L = {"W1": [normal(Fs, H, std=0.02) for _ in range(T)], "b1": [torch.zeros(Fs, **bf) for _ in range(T)],
                 "W2": [normal(H, Fs, std=0.02) for _ in range(T)], "b2": torch.zeros(H, **bf),
                 "gain": torch.full((H,), 0.5, **bf), "post_w": torch.ones(H, **bf)}
            L["dW1"], L["dW2"] = [own(w, 0.01) for w in L["W1"]], [own(w, 0.01) for w in L["W2"]]
            L["db1"], L["db2"] = [own(b) for b in L["b1"]], own(L["b2"])
            L["dgain"], L["dpost_w"] = own(L["gain"]), own(L["post_w"])
            L.update(pre=[torch.empty(M, Fs, **bf) for _ in range(T)], A=[torch.empty(M, Fs, **bf) for _ in range(T)],
                     n=torch.empty(M, H, **bf), f=torch.empty(M, H, **bf), y=torch.empty(M, H, **bf),
                     stats=torch.empty(M, 4, **f32))
            self.layers.append(L)
        self.out, self.first_stats = torch.empty(M, H, **bf), torch.empty(M, 4, **f32)
        self.dn, self.dy, self.df = (torch.empty(M, H, **bf) for _ in range(3))
        self.mlp_ws = tp.alloc_workspace(self.mlp.workspace_bytes())
        self.norm_ws = tp.alloc_workspace(self.join.workspace_bytes())
        self.loss = torch.zeros((), **f32)
        self.opt = tp.TPAdamW(params, grads, state_bits=state_bits, weight_decay=decay, beta2=0.99, seed=seed)

    def forward(self):
        L = self.layers
        self.first.fwd(self.x, pre_w=self.norm_w[0], N=L[0]["n"], stats=self.first_stats)
        x = self.x
        for i, l in enumerate(L):
            self.mlp.fwd([l["n"]], l["W1"], l["b1"], l["W2"], l["b2"], [l["f"]], l["pre"], l["A"],
                         workspace=self.mlp_ws)
            n = L[i + 1]["n"] if i + 1 < len(L) else self.out
            self.join.fwd(x, l["f"], l["gain"], l["post_w"], None, self.norm_w[i + 1], None, l["y"], n,
                          stats=l["stats"])
            x = l["y"]
        diff = self.out.float() - self.target.float()
        self.loss.copy_(diff.square().mean())
        self.dn.copy_(diff * (2.0 / diff.numel()))

    def backward(self):
        dy = None  # past the output's norm nothing takes the stream
        for i in reversed(range(len(self.layers))):
            l = self.layers[i]
            self.join.bwd(dy, self.dn, l["y"], l["f"], l["gain"], l["post_w"], None, self.norm_w[i + 1], l["stats"],
                          self.dy, self.df, l["dgain"], l["dpost_w"], None, self.d_norm_w[i + 1], None,
                          workspace=self.norm_ws)
            dy = self.dy
            self.mlp.bwd([self.df], [l["n"]], l["W1"], l["W2"], l["pre"], l["A"], [self.dn], l["dW1"], l["db1"],
                         l["dW2"], l["db2"], self.mlp_ws)
        self.first.bwd(dy, self.dn, self.x, None, None, None, None, self.norm_w[0], self.first_stats, self.dy, None,
                       None, None, None, self.d_norm_w[0], None, workspace=self.norm_ws)

    def step(self):
        self.forward()
        self.backward()
        self.opt.grad_norm(max_norm=1.0)
        self.opt.step(self.lr)

    def capture(self):
        """The whole step as a CUDA graph; replaying it is taking a step."""
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--blocks", type=int, default=3)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    stack = BlockStack(blocks=a.blocks, state_bits=a.state_bits)
    stack.step()  # the first step loads the kernels
    graph = stack.capture()
    for k in range(1, a.steps):
        graph.replay()
        if k % 10 == 9:
            print(f"step {int(stack.opt.steps):4d}  loss {float(stack.loss):.4f}  "
                  f"gradient norm {float(stack.opt.norm):.4f}")


if __name__ == "__main__":
    main()
