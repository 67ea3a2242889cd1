"""The rotary embedding (CUDA) against the float64 oracle.

Tolerance: cos and sin are off by at most 2^-21 (the angle's fraction of a turn is rounded to fp32
at most half a turn, 2^-25 turns = 2 pi 2^-25 radians, and sincospif adds 2 units of 2^-24), the
rotated pair's two products and sum by three roundings, all relative to the pair's length r:
2^-20 r, and one rounding of the result, 2^-8 |y| for bf16.
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


def rand(shape, dtype, seed=0):
    return torch.from_numpy(np.random.default_rng([seed, *shape]).standard_normal(shape, dtype=np.float32)).to(DT[dtype]).cuda()


def check(got, x, pos, split, dtype, theta=1e4, inverse=False):
    x64 = x.double().cpu().numpy()
    want = od.rope(x64, pos, split, theta, inverse)
    m = sum(split)
    r = np.hypot(x64[..., 0:m:2], x64[..., 1:m:2]).repeat(2, axis=-1)
    tol = np.zeros_like(want)
    tol[..., :m] = 2.0 ** -20 * r + (2.0 ** -8 * abs(want[..., :m]) if dtype == "bf16" else 0)
    err = abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), np.argwhere(err > tol)[:5]


SPLITS = [(32, (8, 12, 12)), (64, (16, 24, 24)), (128, (32, 48, 48)), (64, (0, 0, 64)), (64, (0, 32, 0)), (32, (2, 2, 2)),
          (40, (6, 14, 20)), (96, (10, 2, 36)), (256, (86, 84, 86)), (8, (0, 0, 0)), (8, (2, 4, 2)), (24, (22, 0, 2))]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,split", SPLITS)
def test_grid_positions(blin, d, split, dtype):
    B, Hq, Hk, T, Hg, Wg, t0 = 2, 3, 2, 3, 5, 7, 4
    q, k = rand((B, Hq, T * Hg * Wg, d), dtype), rand((B, Hk, T * Hg * Wg, d), dtype, 1)
    pos = od.rope_positions(T, Hg, Wg, t0)
    for inverse in (False, True):
        qr, kr = blin.rope(q, k, grid=(T, Hg, Wg), t0=t0, rope_split=split, inverse=inverse)
        check(qr, q, pos, split, dtype, inverse=inverse)
        check(kr, k, pos, split, dtype, inverse=inverse)
    assert torch.equal(blin.rope(q, grid=(T, Hg, Wg), t0=t0, rope_split=split, inverse=True), qr)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N", [(1, 1), (64, 1), (3, 33), (1, 2000)])
def test_given_positions(blin, B, N, dtype):
    """Positions of any size and sign, per batch row and shared."""
    split = (16, 24, 16)
    rng = np.random.default_rng([B, N])
    pos = rng.integers(-100, 200000, (B, N, 3))
    pos.reshape(-1, 3)[0] = (2 ** 31 - 1, -2 ** 31, 12345678)
    pt = torch.from_numpy(pos.astype(np.int32)).cuda()
    q, k = rand((B, 4, N, 64), dtype), rand((B, 1, N, 64), dtype, 1)
    qr, kr = blin.rope(q, k, positions=pt, rope_split=split, theta=5e5)
    check(qr, q, pos, split, dtype, 5e5)
    check(kr, k, pos, split, dtype, 5e5)
    qs = blin.rope(q, positions=pt[0].contiguous(), rope_split=split, theta=5e5)
    check(qs, q, pos[0], split, dtype, 5e5)


def test_agrees_with_the_rotation_inside_prefill(blin):
    """One-token blocks and a single token: prefill's numerator is (R phi(q)) . (R phi(k)) v, so with
    tokens 0 and 1 its second row follows from rope() by hand."""
    d, split = 32, (8, 12, 12)
    q, k, v = (rand((1, 2, 2, d), "f32", i).abs() for i in range(3))
    o = blin.prefill(q, k, v, grid=(1, 1, 2), block_frames=1, rope_split=split, eps=0.5)
    qr, kr = blin.rope(q, k, grid=(1, 1, 2), rope_split=split)
    num = (qr @ kr.mT) @ v
    den = (q * k.sum(dim=2, keepdim=True)).sum(-1, keepdim=True) + 0.5
    torch.testing.assert_close(o, num / den, rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_strided_and_special_values(blin, dtype):
    B, H, N, d, split = 2, 3, 70, 64, (16, 16, 16)
    fused = rand((B, N, 3, H, d), dtype)
    fused[0, 0, 0, 0, 50:] = float("nan")  # features past the split are copied bit for bit
    fused[0, 1, 0, 0, 0], fused[0, 1, 0, 0, 1] = float("inf"), 1.0  # an infinity stays in its pair
    q, k = fused[:, :, 0].transpose(1, 2), fused[:, :, 1].transpose(1, 2)
    qc, kc, rest = q.contiguous(), k.contiguous(), fused[:, :, 2].clone()
    want = blin.rope(qc, kc, grid=(7, 2, 5), rope_split=split)
    got = blin.rope(q, k, grid=(7, 2, 5), rope_split=split)
    outs = blin.rope(q, k, grid=(7, 2, 5), rope_split=split, out=(q, k))  # in place, strided
    assert outs[0] is q and outs[1] is k
    view = lambda t: t.contiguous().view(torch.int16 if dtype == "bf16" else torch.int32)
    for w, g, o in zip(want, got, outs):
        assert torch.equal(view(w), view(g)) and torch.equal(view(w), view(o))
    assert torch.equal(fused[:, :, 2], rest)
    assert torch.isnan(want[0][0, 0, 0, 50:]).all() and torch.isfinite(want[0][0, 0, 0, :48]).all()
    assert torch.isfinite(want[0][0, 0, 1, 2:]).all() and not torch.isfinite(want[0][0, 0, 1, 0])


def test_gradient(blin):
    """The inverse rotation takes the gradient back: against central differences of the forward."""
    B, H, N, d, split = 1, 2, 5, 32, (8, 12, 10)
    x, g = rand((B, H, N, d), "f32"), rand((B, H, N, d), "f32", 1)
    grid = (1, 1, 5)
    grad = blin.rope(g, grid=grid, t0=9, rope_split=split, inverse=True)
    for idx in [(0, 0, 0, 0), (0, 1, 4, 9), (0, 0, 3, 29), (0, 1, 2, 31)]:
        e = torch.zeros_like(x)
        e[idx] = 0.5  # the map is linear: any step is exact up to rounding
        up, dn = (blin.rope(x + s * e, grid=grid, t0=9, rope_split=split).double() for s in (1, -1))
        diff = (g.double() * (up - dn)).sum().item()
        # 2 x 64 products of about 1, each to 2^-20 of its pair's length (at most 4 here)
        assert abs(diff - grad[idx].item()) <= 128 * 4 * 2.0 ** -20


def test_many_heads_and_streams(blin):
    q = rand((1, 300, 3, 32), "bf16")
    want = blin.rope(q, grid=(3, 1, 1), rope_split=(8, 12, 12))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = blin.rope(q, grid=(3, 1, 1), rope_split=(8, 12, 12), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    check(want, q, od.rope_positions(3, 1, 1), (8, 12, 12), "bf16")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        og = blin.rope(q, grid=(3, 1, 1), rope_split=(8, 12, 12))
    g.replay()
    assert torch.equal(og, want)


def test_the_binding_refuses(blin):
    q = rand((1, 2, 6, 32), "bf16")
    kw = dict(rope_split=(8, 12, 12))
    with pytest.raises(ValueError, match="either"):
        blin.rope(q, **kw)
    pos = torch.zeros(1, 6, 3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="either"):
        blin.rope(q, grid=(1, 2, 3), positions=pos, **kw)
    for bad in (pos.long(), pos[:, :5], pos.cpu(), pos.transpose(1, 2)):
        with pytest.raises(ValueError):
            blin.rope(q, positions=bad, **kw)
    with pytest.raises(ValueError):
        blin.rope(q, q.float(), grid=(1, 2, 3), **kw)
    buf = rand((1, 2, 7, 32), "bf16")
    with pytest.raises(ValueError, match="overlap"):
        blin.rope(q, q.clone(), grid=(1, 2, 3), out=(q.clone(), q), **kw)
    with pytest.raises(ValueError, match="overlap"):  # in place but shifted
        flat = buf.view(-1)
        blin.rope(flat[:384].view(1, 2, 6, 32), grid=(1, 2, 3), out=flat[32:416].view(1, 2, 6, 32), **kw)
    with pytest.raises(blin.BlinError, match="SHAPE"):
        blin.rope(q, grid=(1, 2, 4), **kw)
    with pytest.raises(blin.BlinError, match="SHAPE"):
        blin.rope(q, grid=(1, 2, 3), rope_split=(8, 12, 14))


def test_arguments_without_a_truth_value_or_an_address(blin):
    q = rand((1, 2, 6, 32), "bf16")
    with pytest.raises(TypeError, match="inverse"):
        blin.rope(q, grid=(1, 2, 3), rope_split=(8, 12, 12), inverse=np.zeros(2))

    class NoAddress:
        cuda_stream = "x"

    with pytest.raises(TypeError, match="stream"):
        blin.rope(q, grid=(1, 2, 3), rope_split=(8, 12, 12), stream=NoAddress())
