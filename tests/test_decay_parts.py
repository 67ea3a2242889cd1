"""Decayed linear attention (CUDA): the order of products, the parts of a carried state and the pieces of a
split prompt, against the recurrence in float64.

Tolerances, with `A` the same sum over absolute values and n 2^-24 A for a chain of n fp32 roundings:
  fp32 outputs   (d + 272) 2^-24 A: at most d + 2 C + 16 roundings a term (C = 128 tokens of a chunk).
  bf16 outputs   on top of that the scores' rounding to bf16, 2^-8 of what the call's own tokens add (A_kv),
                 the second bf16 part of the state, 2^-8 of a rest that is 2^-8 of the state: 2^-16 of what
                 the state adds, and the result's own rounding, 2^-8 |o|.
  states         C + 3 roundings a chunk of terms whose weights are exact to 2^-22: 2^-17 S_A elementwise,
                 2e-6 in the 2-norm (unrelated roundings).
"""
import numpy as np
import pytest
import torch

from oracle import decay as od

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def blin():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import block_causal_linear_rope_b200 as m
    yield m
    assert m.device_status() == 0


def recurrence(q, k, v, lg, scale, S):
    """(o, S) of q, k, v [H, N, d], finite log decays and entering states [H, d, d] in float64, 64 tokens at a time."""
    q, k, v, lg, S = (x.double() for x in (q, k, v, lg, S))
    H, N, d = q.shape
    g = lg.view(H, 1, 1)
    o = torch.empty_like(q)
    for a in range(0, N, 64):
        x, y, z = (t[:, a:a + 64] for t in (q, k, v))
        i = torch.arange(x.shape[1], device=q.device, dtype=torch.float64)
        far = (i.view(-1, 1) - i).clamp(min=0)
        w = torch.where(i.view(-1, 1) >= i, torch.exp(g * far), 0.0)
        o[:, a:a + 64] = scale * ((x @ y.mT * w) @ z + torch.exp(g * (i.view(1, -1, 1) + 1)) * (x @ S))
        left = (i[-1] - i).view(1, -1, 1)
        S = torch.exp(g * len(i)) * S + (torch.exp(g * left) * y).mT @ z
    return o, S


def test_the_float64_chunks_are_the_oracle():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 1, 3, 150, 8))
    S0, lg = rng.standard_normal((1, 3, 8, 8)), np.array([0.0, -0.02, -7.0])
    o, S = od.decay_attention(q, k, v, lg, 0.3, S0)
    mine, mineS = recurrence(*(torch.from_numpy(x[0]) for x in (q, k, v)), torch.from_numpy(lg), 0.3, torch.from_numpy(S0[0]))
    np.testing.assert_allclose(mine.numpy(), o[0], rtol=1e-11, atol=1e-11)
    np.testing.assert_allclose(mineS.numpy(), S[0], rtol=1e-11, atol=1e-11)


def inputs(B, H, N, d, dtype, seed, slots=None, size=1.0):
    """q, k, v (k and v of the given size), a pool of states and log decays."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v = (torch.randn(B, H, N, d, generator=gen, device="cuda") for _ in range(3))
    pool = torch.randn(slots or B, H, d, d, generator=gen, device="cuda")
    lg = torch.tensor([-0.0007, -0.02, 0.0, -0.3, -0.004], device="cuda").repeat(-(-H // 5))[:H].contiguous()
    return [q.to(DT[dtype]), (size * k).to(DT[dtype]), (size * v).to(DT[dtype])], pool, lg


def check_row(o, S1, q, k, v, lg, scale, S0, dtype, label):
    """One batch row's outputs and final state against the recurrence."""
    d = q.shape[-1]
    want, S = recurrence(q, k, v, lg, scale, S0)
    nil = torch.zeros_like(S0)
    A_kv, S_kv = recurrence(q.abs(), k.abs(), v.abs(), lg, abs(scale), nil)
    A_S, S_S = recurrence(q.abs(), nil[:, :1, :].expand_as(k), nil[:, :1, :].expand_as(v), lg, abs(scale), S0.abs())
    tol = (d + 272) * 2.0 ** -24 * (A_kv + A_S)
    if dtype == "bf16":
        # an old token's share comes by way of the state: its second part's rounding is below the scores'
        tol = tol + 2.0 ** -8 * (A_kv + want.abs()) + 2.0 ** -16 * A_S
    err = (o.double() - want).abs()
    assert (err <= tol).all(), (label, (err - tol).max().item(), (err > tol).nonzero()[:4].tolist())
    err = (S1.double() - S).abs()
    assert (err <= 2.0 ** -17 * (S_kv + S_S)).all(), label
    assert err.norm() <= 2e-6 * S.norm(), (label, (err.norm() / S.norm()).item())


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64, 128])
def test_repeated_prompts_have_equal_bits(blin, d):
    """Many chunks per CTA, all SMs busy: each chunk's products go over operands and sums of the chunk
    before, and a product that overtook another would show as bits that differ from run to run."""
    B, H, N, dtype = 4, 75, 1700, "bf16"
    (q, k, v), pool, lg = inputs(B, H, N, d, dtype, 1)
    assert blin.decay_workspace_size(B, H, N, d, DT[dtype]) == 16  # one CTA walks a whole prompt
    ref_pool = pool.clone()
    ref = blin.decay_prefill(q, k, v, lg, state=ref_pool, scale=d ** -0.5)
    for _ in range(20):
        p = pool.clone()
        assert torch.equal(blin.decay_prefill(q, k, v, lg, state=p, scale=d ** -0.5), ref) and torch.equal(p, ref_pool)
    for b in range(B):
        check_row(ref[b], ref_pool[b], q[b], k[b], v[b], lg, d ** -0.5, pool[b], dtype, b)
