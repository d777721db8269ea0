"""Group norm in float64 and limits of its error in the root mean square of a whole output.

The element-wise bounds of test_group_norm_gpu.py allow every rounding of a long sum to point one
way.  Here: an element of an fp32 output is the work of at most 64 roundings of half a step (the
sums of its mean and variance are trees some 20 deep over runs of at most some 100 values whose
roundings are independent, a root, an exponential and a quotient of a few steps, some ten products
and sums): 2^-18 of the output's size.  A bf16 output is rounded once more, 2^-8 / sqrt(3) in the root mean square
at the most.  A sum over m samples and positions adds sqrt(m) independent roundings of 2^-24.
Where a mean is 1000 deviations, a run of 100 sums is off by 2^-24 / sqrt(3) sqrt(100 / 3) of it, and the
20 levels of the tree by 2^-24 / sqrt(3) sqrt(20): 2.6e-4 deviations, held to 2^-10 of a deviation.
"""
import torch

EPS = 1e-5
ACT = {"none": lambda t: t, "silu": lambda t: t * torch.sigmoid(t), "sigmoid": torch.sigmoid}


def limit(dtype, sums=0):
    own = 1.1 * 2.0 ** -8 / 3 ** 0.5 if dtype == torch.bfloat16 else 0.0
    return own + 2.0 ** -18 + 2.0 ** -24 * sums ** 0.5


def rms(got, want):
    return float((got.double() - want).norm() / want.norm())


def model(x, dy, G, w, b, gate, act):
    """The outputs and gradients, by name."""
    leaf = {n: t.double().requires_grad_() for n, t in dict(x=x, weight=w, bias=b, gate=gate).items() if t is not None}
    h = leaf["x"].reshape(x.shape[0], -1, G, x.shape[-1] // G)
    mean = h.mean(dim=(1, 3))
    rstd = (h.var(dim=(1, 3), unbiased=False) + EPS).rsqrt()
    z = ((h - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape) * leaf["weight"] + leaf["bias"]
    y = ACT[act](z) if gate is None else z * ACT[act](leaf["gate"])
    y.backward(dy.double())
    return {"y": y.detach(), "mean": mean.detach(), "rstd": rstd.detach(), **{"d" + n: t.grad for n, t in leaf.items()}}


def inputs(shape, dtype, seed, gate, mean=0.3, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *s, m=0.0, sd=1.0: torch.empty(s).normal_(m, sd, generator=gen).to(device)  # noqa: E731
    C = shape[-1]
    return dict(x=normal(*shape, m=mean).to(dtype), dy=normal(*shape).to(dtype), w=normal(C, m=1.0, sd=0.2), b=normal(C, sd=0.2),
                gate=normal(*shape).to(dtype) if gate else None)
