"""Decayed linear attention (CUDA) against the float64 oracle.

Tolerances.  Every output is a sum of products; with `A` the same sum over absolute values
(the oracle on |q|, |k|, |v|), a chain of n fp32 roundings is off by at most n 2^-24 A.
  fp32: at most d + 2 C + 16 roundings a term (C = 128 tokens of a chunk): (d + 272) 2^-24 A.
  bf16 outputs: scores are rounded to bf16 for the tensor cores (the state to two bf16 parts, 2^-16)
    and the result once more, each by at most 2^-8 of the rounded value: 2^-8 (A + |o|) on top of the
    fp32 bound holds for any share of the state (test_decay_parts bounds that share closely).  As
    these roundings are unrelated, their 2-norms add in quadrature: below 2^-8 of the output's (each
    rounding's is about 2^-8 / sqrt(3) of what it rounds, and the two parts are no larger than the
    sum where they are unrelated); twice that is allowed.
  states (fp32 whatever the inputs): (N-independent, as old terms decay with the state)
    C + 3 roundings a chunk of terms whose weights are exact to 2^-22: 2^-17 S_A elementwise with
    S_A the state of absolute values, and 2e-6 in the 2-norm (unrelated roundings).
"""
import numpy as np
import pytest
import torch

from oracle import decay as od

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def blin():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import block_causal_linear_rope_b200 as m
    yield m
    assert m.device_status() == 0


def inputs(B, H, N, d, dtype, seed=0, slots=None):
    """q, k, v, the pool and log decays from 0 to fast ones, as tensors and as float64 arrays."""
    rng = np.random.default_rng([seed, B, H, N, d])
    qkv = [torch.from_numpy(rng.standard_normal((B, H, N, d), dtype=np.float32)).to(DT[dtype]).cuda() for _ in range(3)]
    pool = torch.from_numpy(rng.standard_normal((slots or B, H, d, d), dtype=np.float32)).cuda()
    decays = np.array([-0.02, 0.0, -0.9, -2.0 ** -10, -7.0, -np.inf, -0.2], np.float32)
    lg = torch.from_numpy(decays[(np.arange(H) + seed) % len(decays)]).cuda()
    return qkv, pool, lg


def f64(t):
    return t.double().cpu().numpy()


def check_out(got, q, k, v, lg, scale, dtype, S=None, lengths=None, label=""):
    want, S1 = od.decay_attention(q, k, v, lg, scale, S, lengths)
    A, SA = od.decay_attention(abs(q), abs(k), abs(v), lg, abs(scale), None if S is None else abs(S), lengths)
    d = q.shape[-1]
    tol = (d + 272) * 2.0 ** -24 * A
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (A + abs(want))
    err = abs(f64(got) - want)
    assert (err <= tol).all(), (label, np.argwhere(err > tol)[:5])
    if dtype == "bf16" and want.size > 4096:
        for h in range(q.shape[1]):  # each head by itself: a fast one must not hide behind a slow one
            assert np.linalg.norm(err[:, h]) <= 2.0 ** -7 * np.linalg.norm(want[:, h]), (label, h)
    return S1, SA


def check_state(got, S1, SA):
    err = abs(f64(got) - S1)
    assert (err <= 2.0 ** -17 * SA).all()
    assert np.linalg.norm(err) <= 2e-6 * np.linalg.norm(S1)


SHAPES = [(1, 1, 1), (2, 3, 2), (1, 2, 63), (1, 7, 64), (2, 2, 65), (1, 3, 127), (1, 2, 128), (1, 2, 129), (3, 1, 300),
          (1, 2, 1025)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("B,H,N", SHAPES)
def test_prompt_matches_oracle(blin, B, H, N, d, dtype):
    (q, k, v), pool, lg = inputs(B, H, N, d, dtype)
    S0 = f64(pool)
    o = blin.decay_prefill(q, k, v, lg, state=pool, scale=d ** -0.5)
    S1, SA = check_out(o, f64(q), f64(k), f64(v), f64(lg), d ** -0.5, dtype, S0)
    check_state(pool, S1, SA)
    # and without a state
    check_out(blin.decay_prefill(q, k, v, lg, scale=-1.5), f64(q), f64(k), f64(v), f64(lg), -1.5, dtype)


def test_long_prompts_in_several_segments(blin):
    for dtype, d, N in (("bf16", 32, 9000), ("bf16", 64, 5000), ("bf16", 128, 4100), ("f32", 64, 3000)):
        (q, k, v), pool, lg = inputs(1, 2, N, d, dtype, seed=3)
        lg = torch.tensor([-0.0005, -0.03], device="cuda")
        assert blin.decay_workspace_size(1, 2, N, d, DT[dtype]) > 16
        S0 = f64(pool)
        o = blin.decay_prefill(q, k, v, lg, state=pool, scale=d ** -0.5)
        S1, SA = check_out(o, f64(q), f64(k), f64(v), f64(lg), d ** -0.5, dtype, S0, label=(dtype, d))
        check_state(pool, S1, SA)


@pytest.mark.parametrize("dtype,d,N", [("bf16", 64, 700), ("bf16", 128, 300), ("bf16", 32, 520), ("f32", 64, 200),
                                       ("f32", 128, 4000)])
def test_ragged_rows_with_nan_behind_them(blin, dtype, d, N):
    """Rows of several lengths, none and all of the tokens; what lies behind a row's end is NaN or
    infinite and must not show; slots are permuted, two rows are idle, other slots stay as they are."""
    B, H, P = 7, 2, 9
    (q, k, v), pool, lg = inputs(B, H, N, d, dtype, seed=1, slots=P)
    L = [N, 0, 1, N // 2, N - 1, 129, 5]
    slots = [4, 7, 0, -1, 8, 2, -5]
    for b, n in enumerate(L):
        q[b, :, n:], k[b, :, n:], v[b, :, n:] = float("nan"), float("inf"), float("nan")
    S0 = f64(pool)
    out = torch.full_like(q, 7.0)
    o = blin.decay_prefill(q, k, v, lg, state=pool, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"),
                           lengths=torch.tensor(L, dtype=torch.int32, device="cuda"), scale=0.25, out=out)
    assert o is out
    after = f64(pool)
    for b, n in enumerate(L):
        if slots[b] < 0:
            assert not o[b].any()
            continue
        assert not o[b, :, n:].any()
        row = [f64(x[b:b + 1, :, :n]) for x in (q, k, v)]
        S1, SA = check_out(o[b:b + 1, :, :n], *row, f64(lg), 0.25, dtype, S0[slots[b]][None], label=b)
        err = abs(after[slots[b]] - S1[0])
        assert (err <= 2.0 ** -17 * SA[0]).all(), b
    for p in set(range(P)) - {s for s in slots if s >= 0}:
        assert (after[p] == S0[p]).all()
    assert (after[7] == S0[7]).all()  # the row of length 0


def test_lengths_are_clamped(blin):
    (q, k, v), pool, lg = inputs(2, 2, 40, 64, "bf16")
    n = torch.tensor([-3, 1000], dtype=torch.int32, device="cuda")
    a, b = pool.clone(), pool.clone()
    o1 = blin.decay_prefill(q, k, v, lg, state=a, lengths=n)
    o2 = blin.decay_prefill(q, k, v, lg, state=b, lengths=torch.tensor([0, 40], dtype=torch.int32, device="cuda"))
    assert torch.equal(o1, o2) and torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 7), (33, 4)])
def test_step_matches_oracle(blin, B, H, d, dtype):
    (q, k, v), pool, lg = inputs(B, H, 1, d, dtype, seed=2)
    S0 = f64(pool)
    o = blin.decay_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], lg, pool, scale=d ** -0.5)
    want, S1 = od.decay_attention(f64(q), f64(k), f64(v), f64(lg), d ** -0.5, S0)
    A, SA = od.decay_attention(abs(f64(q)), abs(f64(k)), abs(f64(v)), f64(lg), d ** -0.5, abs(S0))
    tol = (d + 8) * 2.0 ** -24 * A[:, :, 0] + (2.0 ** -8 * abs(want[:, :, 0]) if dtype == "bf16" else 0)
    assert (abs(f64(o) - want[:, :, 0]) <= tol).all()
    assert (abs(f64(pool) - S1) <= 4 * 2.0 ** -24 * SA).all()  # decay, product and sum: three roundings, and the decay's own


def test_step_slots(blin):
    B, H, d, P = 5, 3, 64, 8
    (q, k, v), pool, lg = inputs(B, H, 1, d, "bf16", seed=4, slots=P)
    slots = [6, -1, 0, 3, -1]
    before = pool.clone()
    dense = pool[[6, 0, 0, 3, 0]].contiguous()
    args = [x[:, :, 0].contiguous() for x in (q, k, v)]
    o = blin.decay_step(*args, lg, pool, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    od_ = blin.decay_step(*args, lg, dense)
    for b, s in enumerate(slots):
        if s < 0:
            assert not o[b].any()
        else:
            assert torch.equal(o[b], od_[b]) and torch.equal(pool[s], dense[b])
    for p in (1, 2, 4, 5, 7):
        assert torch.equal(pool[p], before[p])


@pytest.mark.parametrize("bad,code", [([2, 9, 0], 64), ([2, 0, 2], 65)])
def test_bad_slots_are_idle_and_reported(blin, bad, code):
    """A slot past the pool, and one named twice (the first row has it): the row's outputs are
    zeros, no state is touched for it, and device_status tells."""
    B, H, d, P = 3, 2, 32, 4
    (q, k, v), pool, lg = inputs(B, H, 70, d, "bf16", seed=5, slots=P)
    slots = torch.tensor(bad, dtype=torch.int32, device="cuda")
    good = slots.clone()
    good[1 if code == 64 else 2] = -1
    ref = pool.clone()
    o = blin.decay_prefill(q, k, v, lg, state=pool, slots=slots)
    assert blin.device_status() == code and blin.device_status() == 0
    assert torch.equal(o, blin.decay_prefill(q, k, v, lg, state=ref, slots=good)) and torch.equal(pool, ref)
    one = [x[:, :, 0].contiguous() for x in (q, k, v)]
    o = blin.decay_step(*one, lg, pool, slots=slots)
    assert blin.device_status() == code
    assert torch.equal(o, blin.decay_step(*one, lg, ref, slots=good)) and torch.equal(pool, ref)
    assert blin.device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_invalid_decays_make_their_head_nan(blin, dtype):
    (q, k, v), pool, lg = inputs(1, 3, 80, 64, dtype, seed=6)
    bad = torch.tensor([-0.1, 0.5, float("nan")], device="cuda")
    o = blin.decay_prefill(q, k, v, bad, state=pool)
    assert torch.isfinite(o[:, 0]).all() and torch.isnan(o[:, 1:]).all()
    assert torch.isfinite(pool[:, 0]).all() and torch.isnan(pool[:, 1:]).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 32), ("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_strided_operands(blin, dtype, d):
    """q, k, v as slices of a fused projection [B, N, 3, H, d], k from elsewhere, o into [B, N, H, d]:
    the bits of the contiguous call."""
    B, H, N = 2, 3, 150
    (q, k, v), pool, lg = inputs(B, H, N, d, dtype, seed=7)
    ref_pool = pool.clone()
    ref = blin.decay_prefill(q, k, v, lg, state=ref_pool)
    fused = torch.empty(B, N, 3, H, d, dtype=DT[dtype], device="cuda")
    fused[:, :, 0], fused[:, :, 2] = q.transpose(1, 2), v.transpose(1, 2)
    fused[:, :, 1] = 0
    wide = torch.full((B, H, N, d + 16), float("nan"), dtype=DT[dtype], device="cuda")
    wide[..., :d] = k
    o = torch.empty(B, N, H, d, dtype=DT[dtype], device="cuda").transpose(1, 2)
    got = blin.decay_prefill(fused[:, :, 0].transpose(1, 2), wide[..., :d], fused[:, :, 2].transpose(1, 2), lg, state=pool,
                             out=o)
    assert got is o and torch.equal(o, ref) and torch.equal(pool, ref_pool)
    a, b = ref_pool.clone(), ref_pool.clone()
    r = blin.decay_step(q[:, :, 3].contiguous(), k[:, :, 3].contiguous(), v[:, :, 3].contiguous(), lg, a)
    s = blin.decay_step(fused[:, 3, 0], wide[:, :, 3, :d], fused[:, 3, 2], lg, b)
    assert torch.equal(r, s) and torch.equal(a, b)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 32)])
def test_a_prompt_and_then_single_tokens(blin, dtype, d):
    """A prompt in two calls and the rest token by token: the oracle's one run over all of it."""
    B, H, N = 2, 3, 200
    (q, k, v), pool, lg = inputs(B, H, N, d, dtype, seed=8)
    S0 = f64(pool)
    parts = [blin.decay_prefill(x[0], x[1], x[2], lg, state=pool, scale=0.5) for x in
             ([t[:, :, a:b] for t in (q, k, v)] for a, b in ((0, 130), (130, 190)))]
    for n in range(190, N):
        parts.append(blin.decay_step(q[:, :, n], k[:, :, n], v[:, :, n], lg, pool, scale=0.5).unsqueeze(2))
    S1, SA = check_out(torch.cat(parts, dim=2), f64(q), f64(k), f64(v), f64(lg), 0.5, dtype, S0)
    check_state(pool, S1, SA)


def test_graph_replay_and_other_streams(blin):
    """A captured step replayed, and a prefill on a side stream with memory made there, give the
    eager calls' bits; runs repeat bit for bit."""
    (q, k, v), pool, lg = inputs(4, 4, 500, 64, "bf16", seed=9)
    start = pool.clone()
    ref = blin.decay_prefill(q, k, v, lg, state=pool)
    ref_pool = pool.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p2 = start.clone()
    side.wait_stream(torch.cuda.current_stream())
    o2 = blin.decay_prefill(q, k, v, lg, state=p2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o2, ref) and torch.equal(p2, ref_pool)
    one = [x[:, :, 5].contiguous() for x in (q, k, v)]
    static = start.clone()
    blin.decay_step(*one, lg, static.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        og = blin.decay_step(*one, lg, static)
        opf = blin.decay_prefill(q, k, v, lg, state=static)
    static.copy_(start)
    eager = start.clone()
    for _ in range(2):
        g.replay()
        oe = blin.decay_step(*one, lg, eager)
        ope = blin.decay_prefill(q, k, v, lg, state=eager)
        assert torch.equal(og, oe) and torch.equal(opf, ope) and torch.equal(static, eager)


def test_the_binding_refuses(blin):
    (q, k, v), pool, lg = inputs(2, 2, 16, 64, "bf16")
    i32 = torch.zeros(2, dtype=torch.int32, device="cuda")
    for kw in (dict(state=pool[:1]), dict(state=pool.bfloat16()), dict(state=pool.cpu()), dict(lengths=i32.long()),
               dict(lengths=i32[:1]), dict(lengths=i32.cpu()), dict(slots=i32), dict(out=q), dict(out=q[:1]),
               dict(out=torch.empty_like(q, dtype=torch.float32))):
        with pytest.raises((ValueError, blin.BlinError)):
            blin.decay_prefill(q, k, v, lg, **kw)
    for args in ((q, k[:1], v, lg), (q, k, v.float(), lg), (q, k, v, lg[:1]), (q, k, v, lg.double()),
                 (q.transpose(2, 3), k.transpose(2, 3), v.transpose(2, 3), lg)):
        with pytest.raises(ValueError):
            blin.decay_prefill(*args)
    x = q[:, :, 0]
    for kw in (dict(out=x), dict(slots=i32.long()), dict(slots=i32[:1])):
        with pytest.raises(ValueError):
            blin.decay_step(x, k[:, :, 0], v[:, :, 0], lg, pool, **kw)
    with pytest.raises(blin.BlinError, match="ALIGN"):
        blin.decay_prefill(*(torch.zeros(1, 1, 8, 68, dtype=torch.bfloat16, device="cuda")[..., 4:] for _ in range(3)), lg[:1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_tokens(blin, dtype):
    q = torch.empty(2, 3, 0, 64, dtype=DT[dtype], device="cuda")
    pool = torch.ones(2, 3, 64, 64, device="cuda")
    assert blin.decay_prefill(q, q, q, torch.zeros(3, device="cuda"), state=pool).shape == q.shape
    assert (pool == 1).all()
    qr, kr = blin.rope(q, q, grid=(0, 2, 2), rope_split=(16, 24, 24))
    assert qr.shape == kr.shape == q.shape


def test_rope_prompt_and_steps_together(blin):
    """As a service runs them: q and k of a fused projection rotated in place over a latent grid, the
    prompt into pool slots, then a single token at a time with given positions; against the oracle
    over the whole sequence.  Each rotated value is off by at most 2^-20 of its pair's length, which
    is at most the sum of the pair's absolute values: 2^-18 A covers both operands of a product."""
    B, H, d, split, grid, extra = 2, 3, 64, (16, 24, 16), (3, 4, 5), 4
    N = grid[0] * grid[1] * grid[2]
    rng = np.random.default_rng(12)
    qkv = rng.standard_normal((B, N + extra, 3, H, d)).astype(np.float32)
    lg = torch.tensor([-0.03, -0.4, 0.0], device="cuda")
    pool = torch.zeros(4, H, d, d, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    fused = torch.from_numpy(qkv[:, :N].copy()).cuda()
    q, k, v = (fused[:, :, i].transpose(1, 2) for i in range(3))
    blin.rope(q, k, grid=grid, t0=2, rope_split=split, out=(q, k))
    outs = [blin.decay_prefill(q, k, v, lg, state=pool, slots=slots, scale=d ** -0.5)]
    pos = list(od.rope_positions(*grid, t0=2))
    for n in range(N, N + extra):
        at = torch.tensor([[n, n, n]], dtype=torch.int32, device="cuda")  # text behind the video
        pos.append(np.array([n, n, n]))
        row = torch.from_numpy(qkv[:, n].copy()).cuda()  # [B, 3, H, d]
        q1, k1 = blin.rope(row[:, 0].unsqueeze(2), row[:, 1].unsqueeze(2), positions=at, rope_split=split)
        outs.append(blin.decay_step(q1.squeeze(2), k1.squeeze(2), row[:, 2], lg, pool, slots=slots,
                                    scale=d ** -0.5).unsqueeze(2))
    x = qkv.transpose(2, 0, 3, 1, 4).astype(np.float64)
    qr, kr = (od.rope(t, np.array(pos), split) for t in x[:2])
    want, S = od.decay_attention(qr, kr, x[2], f64(lg), d ** -0.5)

    def lengths(t):  # each feature's bound: its pair's absolute sum
        y = abs(t).reshape(*t.shape[:-1], -1, 2)
        return (y.sum(-1, keepdims=True) + 0 * y).reshape(t.shape)

    A, SA = od.decay_attention(lengths(x[0]), lengths(x[1]), abs(x[2]), f64(lg), d ** -0.5)
    assert (abs(f64(torch.cat(outs, dim=2)) - want) <= (2.0 ** -18 + (d + 272) * 2.0 ** -24) * A).all()
    got = f64(pool)
    assert (abs(got[[3, 1]] - S) <= 2.0 ** -17 * SA).all() and not got[[0, 2]].any()


@pytest.mark.parametrize("dtype,d,C,at", [("bf16", 32, 128, 300), ("bf16", 64, 128, 640), ("bf16", 128, 128, 511),
                                          ("f32", 64, 64, 130)])
@pytest.mark.parametrize("where,value", [("k", float("nan")), ("v", float("nan")), ("v", float("-inf"))])
def test_a_token_that_is_not_finite_stays_in_its_head(blin, dtype, d, C, at, where, value):
    """One bad key or value: from its token on the head's outputs (a value: those of its feature) are
    not finite, the chunks before it, the other features, heads and rows keep their bits."""
    B, H, N = 2, 3, 700
    (q, k, v), pool, lg = inputs(B, H, N, d, dtype, seed=13)
    lg = torch.full_like(lg, -0.001)
    ref_pool = pool.clone()
    ref = blin.decay_prefill(q, k, v, lg, state=ref_pool)
    (k if where == "k" else v)[1, 2, at, 5] = value
    o = blin.decay_prefill(q, k, v, lg, state=pool)
    bad = o[1, 2] if where == "k" else o[1, 2, :, 5]
    assert not torch.isfinite(bad[at:]).any()
    state = pool[1, 2, 5] if where == "k" else pool[1, 2, :, 5]
    assert not torch.isfinite(state).any()
    first = at // C * C
    assert torch.equal(o[1, 2, :first], ref[1, 2, :first])
    if where == "v":
        rest = [f for f in range(d) if f != 5]
        assert torch.equal(o[1, 2][:, rest], ref[1, 2][:, rest]) and torch.equal(pool[1, 2][:, rest], ref_pool[1, 2][:, rest])
    for b, h in [(b, h) for b in range(B) for h in range(H) if (b, h) != (1, 2)]:
        assert torch.equal(o[b, h], ref[b, h]) and torch.equal(pool[b, h], ref_pool[b, h])


def test_memory_made_for_a_call_belongs_to_its_stream(blin):
    """Work queued on the current stream still writes to memory that has been freed there; a call on
    another stream, which does not wait for it, must not be given that memory."""
    (q, k, v), _, lg = inputs(1, 2, 4096, 64, "bf16", seed=14)
    need = blin.decay_workspace_size(1, 2, 4096, 64)
    assert need > 1 << 16
    want = blin.decay_prefill(q, k, v, lg)
    rot = blin.rope(q, grid=(4096, 1, 1), rope_split=(16, 24, 24))
    x = torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    late = [torch.empty_like(q) for _ in range(4)] + [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for _ in range(30):
        torch.matmul(x, x, out=y)
    for t in late:
        t.fill_(7)
    del late, t
    o = blin.decay_prefill(q, k, v, lg, stream=side)
    r = blin.rope(q, grid=(4096, 1, 1), rope_split=(16, 24, 24), stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(r, rot)


@pytest.mark.parametrize("dtype,d", [("bf16", 32), ("bf16", 64), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("B,H", [(50, 7), (64, 6), (65, 6)])
def test_many_rows_of_unequal_lengths(blin, B, H, d, dtype):
    """More blocks than run at a time: each row's results whatever order the rows are taken in."""
    N, P = 140, B + 3
    (q, k, v), pool, lg = inputs(B, H, N, d, dtype, seed=15, slots=P)
    rng = np.random.default_rng([16, B, d])
    L = rng.integers(0, N + 1, B)
    L[rng.permutation(B)[:9]] = [0, 0, N, N, 64, 64, 64, 1, 128]
    slots = rng.permutation(P)[:B]
    slots[rng.permutation(B)[:3]] = -1
    S0 = f64(pool)
    o = blin.decay_prefill(q, k, v, lg, state=pool, slots=torch.from_numpy(slots.astype(np.int32)).cuda(),
                           lengths=torch.from_numpy(L.astype(np.int32)).cuda(), scale=0.25)
    after = f64(pool)
    live = slots >= 0
    assert not o[torch.from_numpy(~live).cuda()].any()
    S1, SA = check_out(o[torch.from_numpy(live).cuda()], *(f64(x)[live] for x in (q, k, v)), f64(lg), 0.25, dtype,
                       S0[slots[live]], L[live])
    assert (abs(after[slots[live]] - S1) <= 2.0 ** -17 * SA).all()
    idle = sorted(set(range(P)) - set(slots[live].tolist()))
    assert (after[idle] == S0[idle]).all()


def test_calls_at_the_same_time_and_on_a_forked_stream_of_a_capture(blin):
    """Split prompts on two streams at once, eager and as two branches of one graph: each has its own
    scratch, and the bits are those of calls one after the other."""
    (q, k, v), pool, lg = inputs(2, 2, 5000, 64, "bf16", seed=17)
    assert blin.decay_workspace_size(2, 2, 5000, 64) > 16
    lg = torch.full_like(lg, -0.01)
    halves = [[x[b:b + 1] for x in (q, k, v)] for b in range(2)]
    start = [pool[b:b + 1].clone() for b in range(2)]
    ref_pool = [p.clone() for p in start]
    ref = [blin.decay_prefill(*halves[b], lg, state=ref_pool[b]) for b in range(2)]
    side = torch.cuda.Stream()

    def both(pools):
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        outs = [blin.decay_prefill(*halves[0], lg, state=pools[0]), blin.decay_prefill(*halves[1], lg, state=pools[1], stream=side)]
        cur.wait_stream(side)
        return outs

    for _ in range(3):
        pools = [p.clone() for p in start]
        outs = both(pools)
        for b in range(2):
            assert torch.equal(outs[b], ref[b]) and torch.equal(pools[b], ref_pool[b])
    static = [p.clone() for p in start]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = both(static)
    for _ in range(2):
        for b in range(2):
            static[b].copy_(start[b])
        g.replay()
        for b in range(2):
            assert torch.equal(outs[b], ref[b]) and torch.equal(static[b], ref_pool[b])
