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


def inputs(B, H, N, d, dtype, seed, slots=None, size=1.0, device="cuda"):
    """q, k, v (k and v of the given size), a pool of states and log decays."""
    gen = torch.Generator(device=device).manual_seed(seed)
    q, k, v = (torch.randn(B, H, N, d, generator=gen, device=device) for _ in range(3))
    pool = torch.randn(slots or B, H, d, d, generator=gen, device=device)
    lg = torch.tensor([-0.0007, -0.02, 0.0, -0.3, -0.004], device=device).repeat(-(-H // 5))[:H].contiguous()
    return [q.to(DT[dtype]), (size * k).to(DT[dtype]), (size * v).to(DT[dtype])], pool, lg


def bounds(q, k, v, lg, scale, S0, dtype):
    """(o, tolerance of o, S, the state of absolute values) of one batch row."""
    d = q.shape[-1]
    want, S = recurrence(q, k, v, lg, scale, S0)
    nil = torch.zeros_like(S0)
    A_kv, S_kv = recurrence(q.abs(), k.abs(), v.abs(), lg, abs(scale), nil)
    A_S, S_S = recurrence(q.abs(), nil[:, :1, :].expand_as(k), nil[:, :1, :].expand_as(v), lg, abs(scale), S0.abs())
    tol = (d + 272) * 2.0 ** -24 * (A_kv + A_S)
    if dtype == "bf16":
        # an old token's share comes by way of the state: its second part's rounding is below the scores'
        tol = tol + 2.0 ** -8 * (A_kv + want.abs()) + 2.0 ** -16 * A_S
    return want, tol, S, S_kv + S_S


def check_row(o, S1, q, k, v, lg, scale, S0, dtype, label):
    """One batch row's outputs and final state against the recurrence."""
    want, tol, S, SA = bounds(q, k, v, lg, scale, S0, dtype)
    err = (o.double() - want).abs()
    assert (err <= tol).all(), (label, (err - tol).max().item(), (err > tol).nonzero()[:4].tolist())
    err = (S1.double() - S).abs()
    assert (err <= 2.0 ** -17 * SA).all(), label
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


TINY = 2.0 ** -10  # keys and values whose tokens add next to nothing to a state of ones: 2^-13 d against d


@pytest.mark.parametrize("d", [32, 64, 128])
def test_the_bound_tells_one_part_of_a_state_from_two(d):
    """The state that multiplies the queries as one bf16, and with a second part that is a chunk of 128 tokens
    old: both break the bound that the next test sets; two parts keep it."""
    (q, k, v), pool, lg = inputs(1, 2, 300, d, "bf16", 2, size=TINY, device="cpu")
    want, tol, _, _ = bounds(q[0], k[0], v[0], lg, d ** -0.5, pool[0], "bf16")
    S, old = pool[0].double(), torch.zeros_like(pool[0]).double()
    ok = {"one": True, "stale": True, "two": True}
    for a in range(0, 300, 128):
        x, y, z = (t[0][:, a:a + 128] for t in (q, k, v))
        hi = S.to(torch.bfloat16).double()
        lo = (S - hi).to(torch.bfloat16).double()
        for name, part in (("one", 0.0 * lo), ("stale", old), ("two", lo)):
            o, _ = recurrence(x, y, z, lg, d ** -0.5, hi + part)
            err = (o.to(torch.bfloat16).double() - want[:, a:a + 128]).abs()
            ok[name] &= bool((err <= tol[:, a:a + 128]).all())
        old = lo
        _, S = recurrence(x, y, z, lg, 1.0, S)
    assert ok == {"one": False, "stale": False, "two": True}


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("N,split", [(600, False), (2000, True)])
def test_outputs_carry_both_parts_of_the_state(blin, N, split, d):
    """Large entering states, keys and values that add next to nothing, decays that change the state from
    chunk to chunk: the outputs are the state's, to their own rounding and 2^-16 of the state."""
    B, H = (7, 40) if not split else (2, 3)
    (q, k, v), pool, lg = inputs(B, H, N, d, "bf16", 3, size=TINY)
    assert (blin.decay_workspace_size(B, H, N, d) > 16) == split
    after = pool.clone()
    o = blin.decay_prefill(q, k, v, lg, state=after, scale=d ** -0.5)
    for b in range(B):
        check_row(o[b], after[b], q[b], k[b], v[b], lg, d ** -0.5, pool[b], "bf16", b)


# shapes that are cut into several segments (`seg` tokens) of several pieces (`piece` tokens), and shapes whose
# rows are also taken longest first, as not all blocks of the second launch start at once
PIECES = [("bf16", 32, 3, 33, 1536, 768, 2, 384), ("bf16", 64, 2, 25, 1536, 768, 2, 384),
          ("bf16", 128, 3, 10, 2176, 768, 4, 384), ("f32", 32, 8, 8, 448, 128, 6, 64), ("f32", 64, 2, 19, 512, 128, 6, 64),
          ("f32", 128, 2, 11, 448, 128, 6, 64)]
SORTED = [("bf16", 32, 10, 30, 9856, 3328, 4, 1664), ("bf16", 64, 5, 30, 9856, 3328, 4, 1664),
          ("bf16", 128, 5, 10, 13952, 2816, 8, 1408), ("f32", 32, 5, 30, 320, 64, 4, 64), ("f32", 64, 10, 10, 320, 64, 4, 64),
          ("f32", 128, 10, 5, 320, 64, 4, 64), ("f32", 64, 20, 3, 576, 64, 8, 64)]
# and shapes of one piece a segment, with fewer rows
PLAIN = [("bf16", 32, 7, 2, 2000, 256, 7, 256), ("bf16", 64, 7, 2, 3000, 384, 7, 384), ("bf16", 128, 7, 2, 2000, 256, 7, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,B,H,N,seg,pieces,piece", PIECES + SORTED + PLAIN)
def test_rows_that_end_anywhere_in_a_split_prompt(blin, dtype, d, B, H, N, seg, pieces, piece):
    """Ragged rows, permuted slots and an idle row through the two launches: rows that end inside, at, before
    and behind the borders of pieces and segments; what lies behind them is NaN."""
    # the split that this test is for: one entering state and `pieces` local ones a head
    assert blin.decay_workspace_size(B, H, N, d, DT[dtype]) == 4 * B * H * (1 + pieces) * d * d
    P = B + 2
    data, pool, lg = inputs(B, H, N, d, dtype, 4, slots=P)
    ends = [N, piece + 1, seg, N - 1, seg + 1, piece, seg - 1, piece - 1, 0, seg + piece // 2, 1, piece // 2]
    ends = [min(n, N) for n in ends]
    rounds = -(-len(ends) // B) if dtype == "f32" or B * H * N < 200000 else 1
    gen = torch.Generator().manual_seed(5)
    for r in range(rounds):
        L = [ends[(r * B + b) % len(ends)] for b in range(B)]
        slots = torch.randperm(P, generator=gen)[:B].tolist()
        if B > 3:
            slots[(2 + r) % B] = -1
        q, k, v = (x.clone() for x in data)
        for b, n in enumerate(L):
            q[b, :, n:], k[b, :, n:], v[b, :, n:] = float("nan"), float("inf"), float("nan")
        after = pool.clone()
        o = blin.decay_prefill(q, k, v, lg, state=after, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"),
                               lengths=torch.tensor(L, dtype=torch.int32, device="cuda"), scale=d ** -0.5)
        for b, n in enumerate(L):
            if slots[b] < 0:
                assert not o[b].any()
                continue
            assert not o[b, :, n:].any(), (r, b)
            if n:
                check_row(o[b, :, :n], after[slots[b]], q[b, :, :n], k[b, :, :n], v[b, :, :n], lg, d ** -0.5,
                          pool[slots[b]], dtype, (r, b, n))
            else:
                assert torch.equal(after[slots[b]], pool[slots[b]])
        for p in set(range(P)) - set(slots):
            assert torch.equal(after[p], pool[p])
