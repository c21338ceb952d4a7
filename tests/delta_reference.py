"""The gated delta rule token by token in 64 bits, and what the tests compare with it."""
from __future__ import annotations

import torch


def reference(q, k, v, g, beta, offsets, initial, scale):
    """Outputs [tokens, heads_v, dim_v] (0 in rows of no sequence) and final states [n, heads_v, dim_k, dim_v], float64,
    on the CPU; differentiable. g may be None."""
    q, k, v, beta = (x.double().cpu() if x.dtype != torch.float64 else x for x in (q, k, v, beta))
    g = None if g is None else (g.double().cpu() if g.dtype != torch.float64 else g)
    share = v.shape[1] // q.shape[1]
    outs, finals = {}, []
    for i in range(len(offsets) - 1):
        s = torch.zeros(v.shape[1], q.shape[2], v.shape[2], dtype=torch.float64) if initial is None else initial[i]
        for t in range(int(offsets[i]), int(offsets[i + 1])):
            kt, qt = k[t].repeat_interleave(share, 0), q[t].repeat_interleave(share, 0)
            if g is not None:
                s = s * torch.exp(g[t])[:, None, None]
            u = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", s, kt))
            s = s + kt[:, :, None] * u[:, None, :]
            outs[t] = scale * torch.einsum("hkv,hk->hv", s, qt)
        finals.append(s)
    zero = torch.zeros(v.shape[1:], dtype=torch.float64)
    o = torch.stack([outs.get(t, zero) for t in range(v.shape[0])]) if v.shape[0] else torch.zeros(v.shape, dtype=torch.float64)
    return o, torch.stack(finals)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tolerance(dtype, what):
    """Largest 2-norm of the error over that of the result.

    16-bit results: the result's own rounding and, on the longest path to one, three operands in one part (the inverse,
    S and dS'), half a step each; the others are in two parts or exact. A gate's gradient sums products of S with dS'
    that cancel, so that its terms' roundings count double. fp32 results, and states from 16-bit inputs: at most six
    products deep, each of sums of up to 256 + 64 terms whose roundings add up like a random walk, sqrt(320) half steps
    of fp32; fp16 states have two-part operands besides, off by 2^-22 each, three deep."""
    if what == "state" or dtype == torch.float32:
        return 6 * 320 ** 0.5 * half_step(torch.float32) + (3 * 2.0 ** -22 if dtype == torch.float16 else 0)
    return (8 if what in ("dg", "dbeta") else 4) * half_step(dtype)


def close(got, want, dtype, what, label=""):
    """The error's 2-norm within tolerance(), and no element off by more than ten times that of max(|it|, the
    root-mean-square element), the most that rows of smaller norm than the average make of it."""
    got, want = got.double().cpu(), want.double().cpu()
    assert got.shape == want.shape, (label, what, got.shape, want.shape)
    if not want.numel():
        return
    tol = tolerance(dtype, what)
    assert torch.isfinite(got).all(), f"{label} {what}: {int((~torch.isfinite(got)).sum())} elements not finite"
    norm, off = want.norm().item(), (got - want).norm().item()
    assert off <= tol * norm + 1e-30, f"{label} {what}: off by {off / max(norm, 1e-300):.3g}, {tol:.3g} allowed"
    rms = norm / want.numel() ** 0.5
    worst = ((got - want).abs() / want.abs().clamp(min=max(rms, 1e-300))).max().item()
    assert worst <= 10 * tol, f"{label} {what}: an element off by {worst:.3g}, {10 * tol:.3g} allowed"


def inputs(seed, lens, hk, hv, dk, dv, dtype, gates=(torch.float32, None), init=True, tail=0, device="cuda"):
    """Unit q and k, normal v, decays of 0 to about -3, beta in (0, 1); `tail` rows behind the last sequence."""
    gen = torch.Generator().manual_seed(seed)
    n = sum(lens) + tail

    def normal(*shape):
        return torch.randn(*shape, generator=gen)

    def unit(*shape):
        return torch.nn.functional.normalize(normal(*shape), dim=-1)

    x = {"q": unit(n, hk, dk), "k": unit(n, hk, dk), "v": normal(n, hv, dv)}
    x = {a: b.to(dtype).to(device) for a, b in x.items()}
    x["g"] = (-torch.rand(hv, generator=gen) ** 3 * 2 * torch.nn.functional.softplus(normal(n, hv))).to(gates[0]).to(device)
    x["beta"] = torch.sigmoid(normal(n, hv)).to(gates[1] or dtype).to(device)
    offsets = torch.tensor([0] + list(lens), dtype=torch.int64).cumsum(0).to(device)
    initial = (0.3 * normal(len(lens), hv, dk, dv)).to(device) if init else None
    return x, offsets, initial
