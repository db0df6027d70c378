"""The gated delta rule from its definition, token by token in 64 bits on CPU
tensors; the tests compare the kernels over a pool of states with it."""
import torch


def rows(T, Hk, Hv, dk, dv, seed, lean=0.4, decay=(0.001, 1.0), beta=(0.05, 0.95)):
    """Rows of a recurrent layer: unit-norm queries and keys (bf16) that point
    partly the same way, values N(0, 1), log decays -exp(uniform) and strengths."""
    g = torch.Generator().manual_seed(seed)
    qk = torch.randn(2, T, Hk, dk, generator=g) + lean * torch.randn(2, 1, Hk, dk, generator=g)
    qk = qk / qk.norm(dim=-1, keepdim=True).clamp(min=1e-30)
    v = torch.randn(T, Hv, dv, generator=g)
    lo, hi = (torch.tensor(x).log() for x in decay)
    gate = -torch.exp(lo + (hi - lo) * torch.rand(T, Hv, generator=g))
    b = beta[0] + (beta[1] - beta[0]) * torch.rand(T, Hv, generator=g)
    return dict(q=qk[0].bfloat16(), k=qk[1].bfloat16(), v=v.bfloat16(), g=gate, beta=b)


def run(state, r, first, last, keep_outputs=True):
    """Tokens first..last-1 of rows `r` from `state` [Hv, dv, dk] (float64):
    the state after them and the outputs [n, Hv, dv]."""
    S = state.double().clone()
    Hv, dv, _ = S.shape
    out = torch.zeros(last - first, Hv, dv, dtype=torch.float64)
    group = Hv // r["k"].shape[1]
    for n, t in enumerate(range(first, last)):
        k = r["k"][t].double().repeat_interleave(group, 0)
        S = S * torch.exp(r["g"][t].double())[:, None, None]
        u = r["beta"][t].double()[:, None] * (r["v"][t].double() - torch.einsum("hvk,hk->hv", S, k))
        S = S + u[:, :, None] * k[:, None, :]
        if keep_outputs:
            out[n] = torch.einsum("hvk,hk->hv", S, r["q"][t].double().repeat_interleave(group, 0))
    return S, out


def on(r, device="cuda"):
    return [r[n].to(device) for n in ("q", "k", "v", "g", "beta")]


def close(got, ref, rel, out_step, what):
    """|got - ref| at most `rel` of the reference's largest value in the row
    (last dimension) and largest size of all, and `out_step` of the value."""
    got, ref = got.double().cpu(), ref.double()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert torch.isfinite(got).all(), what + ": not finite"
    if not ref.numel():
        return
    tol = rel * ref.abs().amax(-1, keepdim=True).clamp(min=rel * float(ref.abs().max())) + out_step * ref.abs()
    off = (got - ref).abs() - tol
    assert float(off.max()) <= 0, f"{what}: off by {float((got - ref).abs().max()):.3e}, {float(off.max()):.3e} beyond"
