"""A state-space mixer layer from this package's operators, run over a prompt and then token by token.

    python examples/mixer_layer.py [--batch 2] [--prompt 512] [--tokens 16] [--model 768] [--inner 1536]

One layer, as a model holds many: input projection in e4m3 -> causal convolution -> selective scan (its steps, B and
C projected from the convolved rows) -> gated norm, written in e4m3 -> output projection. The prompt goes through the
layer in one call per operator and leaves two caches per sequence (the convolution's last inputs and the scan's
state); every further token advances them in place. The tokens' outputs are compared with those of one prompt over
everything.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mamba_ssd_prefill_gb300 as ssd  # noqa: E402


class Mixer:
    """Weights of one layer: projections in e4m3 with 128 x 128 block scales, the rest in bf16 and fp32."""

    def __init__(self, model, inner, states=16, width=4, groups=1, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def randn(*shape, scale=1.0):
            return torch.randn(*shape, generator=g, device="cuda") * scale

        self.inner, self.states, self.groups = inner, states, groups
        self.rank = -(-model // 16)
        self.in_proj = ssd.ssd_fp8_quantize(randn(2 * inner, model, scale=model ** -0.5), 128)
        self.out_proj = ssd.ssd_fp8_quantize(randn(model, inner, scale=inner ** -0.5), 128)
        self.conv_weight, self.conv_bias = randn(inner, width, scale=width ** -0.5), randn(inner, scale=0.1)
        self.x_proj = randn(self.rank + 2 * states, inner, scale=inner ** -0.5).bfloat16()
        self.dt_proj = randn(inner, self.rank, scale=self.rank ** -0.5).bfloat16()
        dt0 = torch.exp(torch.rand(inner, generator=g, device="cuda") * math.log(100) + math.log(1e-3))
        self.dt_bias = torch.log(torch.expm1(dt0))  # softplus(dt_bias) is spread over 0.001 .. 0.1
        self.A = -torch.arange(1, states + 1, device="cuda", dtype=torch.float32).repeat(inner, 1)
        self.D = torch.ones(inner, device="cuda")
        self.norm_weight = 1 + randn(inner, scale=0.1)

    def caches(self, batch):
        """(convolution cache, scan states) of new sequences."""
        return (torch.zeros(batch, self.inner, self.conv_weight.shape[1] - 1, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(batch, self.inner, self.states, device="cuda"))

    def __call__(self, hidden, caches):
        """hidden [batch, L, model] (L 1 for single tokens) -> the same shape; the caches advance in place."""
        cache, state = caches
        xz = ssd.ssd_fp8_matmul(*ssd.ssd_fp8_quantize(hidden), *self.in_proj)
        x, z = xz.split(self.inner, -1)  # column slices: the operators read them where they lie
        x, _ = ssd.ssd_conv(x, self.conv_weight, self.conv_bias, cache, conv_state_out=cache)
        low, B, C = (x @ self.x_proj.t()).split([self.rank, self.states, self.states], -1)
        dt = low @ self.dt_proj.t()
        y, _ = ssd.ssd_selective_scan(x, dt, self.dt_bias, self.A, B.unsqueeze(2), C.unsqueeze(2), self.D,
                                      init_states=state, final_states=state)
        y = ssd.ssd_group_norm(y, self.norm_weight, z=z, ngroups=self.groups, gate_first=True, quantize=True)
        return ssd.ssd_fp8_matmul(*y, *self.out_proj)


def run(batch=2, prompt=512, tokens=16, model=768, inner=1536, groups=1, seed=0):
    """Largest relative difference (2-norm) between the tokens' outputs and the same rows of one long prompt."""
    layer = Mixer(model, inner, groups=groups, seed=seed)
    g = torch.Generator("cuda").manual_seed(seed + 1)
    hidden = torch.randn(batch, prompt + tokens, model, generator=g, device="cuda").bfloat16()
    want = layer(hidden, layer.caches(batch))
    caches = layer.caches(batch)
    got = [layer(hidden[:, :prompt].contiguous(), caches)]
    for t in range(prompt, prompt + tokens):
        got.append(layer(hidden[:, t:t + 1].contiguous(), caches))
    got, want = torch.cat(got, 1).float(), want.float()
    return float(((got - want).norm(dim=-1) / want.norm(dim=-1)).max())


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("batch", 2), ("prompt", 512), ("tokens", 16), ("model", 768), ("inner", 1536), ("groups", 1)):
        ap.add_argument(f"--{name}", type=int, default=value)
    args = vars(ap.parse_args())
    print(f"prompt + tokens against one prompt: largest relative difference of a row {run(**args):.2e}")


if __name__ == "__main__":
    main()
