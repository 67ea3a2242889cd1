"""Decayed attention and rotary embedding: host-side refusals (no GPU: every call here is refused
by a host check before any device work, the addresses are never dereferenced)."""
import ctypes

import pytest
import torch

import block_causal_linear_rope_b200 as blin

OK, INVALID, SHAPE, DTYPE, ALIGN, WORKSPACE, STATE = 0, -1, -2, -3, -4, -5, -6
FAKE = 1 << 20


def lay(tok=64, head=0, batch=0, N=8, H=2, d=64):
    return blin.Layout(tok, head or N * d, batch or H * N * d)


def prefill(q=FAKE, k=2 * FAKE, v=3 * FAKE, o=4 * FAKE, dt=1, B=1, H=2, N=8, d=64, lg=FAKE, scale=1.0, layouts=None,
            lengths=None, S=None, slots=0, slot_of=None, ws=None, wb=0):
    return blin.lib.blin_decay_prefill(q, k, v, o, dt, B, H, N, d, lg, scale,
                                       None if layouts is None else ctypes.byref(layouts), lengths, S, slots, slot_of,
                                       ws, wb, None)


def step(q=FAKE, k=2 * FAKE, v=3 * FAKE, o=4 * FAKE, dt=1, B=2, H=2, d=64, lg=FAKE, scale=1.0, layouts=None,
         S=5 * FAKE, slots=2, slot_of=None):
    return blin.lib.blin_decay_step(q, k, v, o, dt, B, H, d, lg, scale,
                                    None if layouts is None else ctypes.byref(layouts), S, slots, slot_of, None)


def check(code, want):
    assert code == want
    assert blin.lib.blin_last_error().decode() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(lg=None), INVALID), (dict(B=0), INVALID), (dict(H=0), INVALID),
    (dict(N=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(d=48), SHAPE), (dict(d=256), SHAPE), (dict(B=1 << 13, H=1 << 12), SHAPE), (dict(N=1 << 30), SHAPE),
    (dict(dt=2), DTYPE), (dict(q=FAKE + 8), ALIGN), (dict(S=FAKE + 4, slots=1), ALIGN), (dict(lg=FAKE + 2), ALIGN),
    (dict(lengths=FAKE + 1), ALIGN), (dict(S=FAKE, slots=1, slot_of=FAKE + 3), ALIGN),
    (dict(S=FAKE, slots=0), STATE), (dict(S=FAKE, slots=3), STATE), (dict(slot_of=FAKE), STATE),
    (dict(o=FAKE), INVALID), (dict(k=4 * FAKE), INVALID),
    (dict(B=1, H=1, N=40000), WORKSPACE), (dict(B=1, H=1, N=40000, ws=FAKE, wb=64), WORKSPACE),
    (dict(B=1, H=1, N=40000, ws=FAKE + 8, wb=1 << 40), ALIGN),
    (dict(layouts=blin.DecayLayouts(lay(), lay(tok=32), lay(), lay())), SHAPE),
    (dict(layouts=blin.DecayLayouts(lay(), lay(), lay(tok=68), lay())), ALIGN),
    (dict(layouts=blin.DecayLayouts(lay(), lay(), lay(), lay(head=8))), SHAPE),
])
def test_prefill_refusals(kw, code):
    check(prefill(**kw), code)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(S=None), INVALID), (dict(slots=0), STATE), (dict(slots=3), STATE), (dict(B=0), INVALID),
    (dict(d=96), SHAPE), (dict(dt=-1), DTYPE), (dict(S=5 * FAKE + 8), ALIGN), (dict(o=2 * FAKE), INVALID),
    (dict(layouts=blin.DecayLayouts(lay(), lay(head=4), lay(), lay())), SHAPE),
])
def test_step_refusals(kw, code):
    check(step(**kw), code)


def test_no_tokens_is_a_no_op():
    assert prefill(N=0) == OK


def test_workspace_sizes():
    ws = blin.lib.blin_decay_workspace_size
    assert ws(1, 2, 8, 64, 1) == 16  # one chunk: one piece
    assert ws(64, 64, 4096, 64, 1) == 16  # heads enough for every SM
    for d in (32, 64, 128):
        n = ws(1, 1, 40000, d, 1)
        assert n > 16 and n % (4 * d * d) == 0 and 2 <= n // (4 * d * d) <= 32
    assert ws(1, 1, 8, 48, 1) == 0 and ws(0, 1, 8, 64, 1) == 0 and ws(1, 1, 8, 64, 5) == 0
    assert blin.decay_workspace_size(1, 2, 8, 64) == 16
    with pytest.raises(ValueError):
        blin.decay_workspace_size(1, 2, 8, 40)


def rope(q=FAKE, qo=2 * FAKE, Hq=2, k=None, ko=None, Hk=0, dt=1, B=1, N=8, d=64, T=2, Hg=2, Wg=2, split=(16, 24, 24),
         theta=1e4, t0=0, pos=None, shared=0, inverse=0, layouts=None, geom=True):
    g = blin._geom(T, Hg, Wg, 1, split, theta, 0.0)
    return blin.lib.blin_rope(q, qo, Hq, k, ko, Hk, dt, B, N, d, ctypes.byref(g) if geom else None, t0, pos, shared, inverse,
                              None if layouts is None else ctypes.byref(layouts), None)


@pytest.mark.parametrize("kw,code", [
    (dict(geom=False), INVALID), (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(k=FAKE, Hk=2), INVALID),
    (dict(k=3 * FAKE, ko=4 * FAKE, Hk=0), INVALID), (dict(Hq=0), INVALID), (dict(B=0), INVALID), (dict(N=-8), INVALID),
    (dict(dt=3), DTYPE), (dict(d=12, split=(4, 4, 4)), SHAPE), (dict(d=264, split=(2, 2, 2)), SHAPE),
    (dict(split=(15, 24, 24)), SHAPE), (dict(split=(-2, 24, 24)), SHAPE), (dict(split=(32, 24, 24)), SHAPE),
    (dict(theta=0.0), INVALID), (dict(theta=float("nan")), INVALID), (dict(inverse=2), INVALID), (dict(shared=-1), INVALID),
    (dict(N=9), SHAPE), (dict(Hg=0), INVALID), (dict(t0=-1), INVALID), (dict(T=-2), INVALID), (dict(t0=1 << 30), SHAPE),
    (dict(q=FAKE + 4), ALIGN), (dict(qo=FAKE + 8), ALIGN), (dict(pos=FAKE + 2), ALIGN),
    (dict(layouts=blin.RopeLayouts(lay(), lay(tok=32), lay(), lay())), SHAPE),
    (dict(layouts=blin.RopeLayouts(lay(tok=68), lay(), lay(), lay())), ALIGN),
    (dict(qo=FAKE, layouts=blin.RopeLayouts(lay(tok=128), lay(tok=64), lay(), lay())), SHAPE),
    (dict(B=1 << 12, Hq=1 << 12), SHAPE),
])
def test_rope_refusals(kw, code):
    check(rope(**kw), code)


def test_rope_without_tokens_is_a_no_op():
    assert rope(N=0, T=0) == OK
    assert rope(N=0, pos=FAKE) == OK


def test_the_binding_refuses_host_tensors_and_wrong_shapes():
    q = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    lg = torch.zeros(2)
    with pytest.raises(TypeError, match="CUDA"):
        blin.decay_prefill(q, q, q, lg)
    with pytest.raises(TypeError, match="CUDA"):
        blin.decay_step(q[:, :, 0], q[:, :, 0], q[:, :, 0], lg, torch.zeros(1, 2, 64, 64))
    with pytest.raises(TypeError, match="CUDA"):
        blin.rope(q, rope_split=(16, 24, 24), grid=(2, 2, 2))
    with pytest.raises(ValueError, match="B, H, N, d"):
        blin.decay_prefill(q[0], q[0], q[0], lg)
    with pytest.raises(ValueError, match="B, H, d"):
        blin.decay_step(q, q, q, lg, torch.zeros(1, 2, 64, 64))
    with pytest.raises(TypeError, match="dtype"):
        blin.decay_prefill(q.half(), q.half(), q.half(), lg)
