"""A layer norm and a linear layer trained and used in 8 bits, by the operators of
dense_gemm_design_amd:

    python examples/fp8_linear.py [--tokens 2048] [--inputs 1024] [--outputs 1536] [--steps 40]

Forward:   h = layer_norm(x);  y = h W^T + b, with h in blocks of 1 x 128 and W in blocks of 128 x 128
Backward:  dh = dy W, dW = dy^T h in e4m3 blocks along what each product sums over (one read of h and
           of dy gives the codes of both their products), the norm's gradients, and all gradients
           clipped by their global norm
Use:       one token at a time through the quantised weights
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_design_amd as dg  # noqa: E402


class NormLinear:
    """fp32 master parameters; products in e4m3 with a scale per block."""

    def __init__(self, inputs, outputs, device, pow2=False, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.pow2 = pow2
        self.gain = torch.ones(inputs, device=device)
        self.shift = torch.zeros(inputs, device=device)
        self.weight = torch.randn(outputs, inputs, generator=g, device=device) * inputs ** -0.5
        self.bias = torch.zeros(outputs, device=device)
        self.requantise()

    @property
    def parameters(self):
        return [self.gain, self.shift, self.weight, self.bias]

    def requantise(self):
        """The weights' codes for y = h W^T and for dh = dy W, after the master weights changed."""
        self.w, self.wt = dg.block_quantize(self.weight, "tile", transposed="both", pow2=self.pow2)

    def forward(self, x):
        h, mean, rstd = dg.layer_norm(x, self.gain, self.shift)
        hq, ht = dg.block_quantize(h, "row", transposed="both", pow2=self.pow2)
        self.held = x, mean, rstd, ht
        return dg.block_gemm(hq, self.w, out_dtype="bf16", bias_col=self.bias)

    def backward(self, dy):
        """Gradients of the parameters, in their order, and of x."""
        x, mean, rstd, ht = self.held
        dyq, dyt = dg.block_quantize(dy, "row", transposed="both", pow2=self.pow2)
        dh = dg.block_gemm(dyq, self.wt, out_dtype="bf16")
        dw = dg.block_gemm(dyt, ht, out_dtype="f32")
        dx, dgain, dshift = dg.layer_norm_backward(dh, x, self.gain, mean, rstd)
        return [dgain, dshift, dw, dy.float().sum(0)], dx

    def token(self, x):
        """y of one token (or a few): no gradients are prepared."""
        h, _, _ = dg.layer_norm(x, self.gain, self.shift)
        return dg.block_gemm(dg.block_quantize(h, pow2=self.pow2), self.w, bias_col=self.bias)


def train(tokens=2048, inputs=1024, outputs=1536, steps=40, pow2=False, rate=0.5, most=1.0,
          device="cuda", say=print):
    """Fits the layer to a random linear map of normalised tokens; returns the losses and the layer."""
    g = torch.Generator(device=device).manual_seed(1)
    x = (torch.randn(tokens, inputs, generator=g, device=device) * 2 + 0.5).to(torch.bfloat16)
    teacher = torch.randn(inputs, outputs, generator=g, device=device) * inputs ** -0.5
    h = torch.nn.functional.layer_norm(x.float(), (inputs,))
    want = h.matmul(teacher) + 0.1
    layer = NormLinear(inputs, outputs, device, pow2)
    losses = []
    for step in range(steps):
        miss = layer.forward(x).float() - want
        losses.append(float(miss.square().mean()))
        grads, _ = layer.backward((miss * (2.0 / tokens)).to(torch.bfloat16))
        norm = dg.clip_grad_norm(grads, most)
        for p, d in zip(layer.parameters, grads):
            p.sub_(d, alpha=rate)
        layer.requantise()
        if say and step % 10 == 0:
            say(f"step {step:3d}  loss {losses[-1]:.5f}  gradient norm {float(norm):.4f}")
    return losses, layer


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    for name, value in (("tokens", 2048), ("inputs", 1024), ("outputs", 1536), ("steps", 40)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--pow2", action="store_true", help="scales that are powers of two")
    a = p.parse_args()
    losses, layer = train(a.tokens, a.inputs, a.outputs, a.steps, a.pow2)
    print(f"loss {losses[0]:.5f} -> {losses[-1]:.5f}")
    x = torch.randn(1, a.inputs, device="cuda").to(torch.bfloat16)
    print("one token:", layer.token(x)[0, :4].tolist())


if __name__ == "__main__":
    main()
