"""What the extension of decay_prefill, decay_step and rope refuses, and what it does for its caller: sizes,
errors, streams, gradients."""
import pytest
import torch

import block_causal_linear_rope_b200 as blin

WIDE = 2 ** 32 + 1  # 1 in 32 bits


def test_dimensions_beyond_32_bits_are_refused():
    """A token count, head count or batch whose low 32 bits name a small problem must not run as that one."""
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    for shape in ((1, 1, WIDE, 64), (1, WIDE, 1, 64), (WIDE, 1, 1, 64)):
        q = x.expand(shape)
        with pytest.raises(ValueError, match="2\\^31"):
            blin.rope(q, grid=(1, 1, 1), rope_split=(16, 24, 24), out=q)
        with pytest.raises(ValueError, match="2\\^31"):
            blin.rope(x, q, grid=(1, 1, 1), rope_split=(16, 24, 24))
        with pytest.raises(ValueError, match="2\\^31"):
            blin.decay_prefill(q, q, q, torch.zeros(1), out=q)
    for shape in ((1, WIDE, 64), (WIDE, 1, 64)):
        q = x[0].expand(shape)
        with pytest.raises(ValueError, match="2\\^31"):
            blin.decay_step(q, q, q, torch.zeros(1), torch.zeros(1, 1, 64, 64), out=q)


def test_workspace_size_of_a_type_that_the_call_does_not_take():
    assert blin.decay_workspace_size(1, 2, 9000, 64, torch.float32) != blin.decay_workspace_size(1, 2, 9000, 64)
    for dtype in (torch.float16, torch.float64, "bf16", None):
        with pytest.raises(TypeError, match="dtype"):
            blin.decay_workspace_size(1, 2, 9000, 64, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_pool_without_slots_is_refused(dtype):
    """Not taken for a call that keeps no state."""
    q = torch.zeros(2, 3, 5, 64, dtype=dtype, device="cuda")
    lg, pool = torch.zeros(3, device="cuda"), torch.zeros(0, 3, 64, 64, device="cuda")
    with pytest.raises(ValueError, match="slots"):
        blin.decay_prefill(q, q, q, lg, state=pool)
    with pytest.raises(ValueError, match="slots"):
        blin.decay_step(q[:, :, 0], q[:, :, 0], q[:, :, 0], lg, pool)


@pytest.mark.gpu
def test_no_memory_for_an_output_is_torchs_error():
    """As of a torch operation: programs that answer it by a smaller batch catch this type."""
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda").expand(1, 4096, 2 ** 24, 64)  # 8 TiB of output
    with pytest.raises(torch.OutOfMemoryError):
        torch.empty(q.shape, dtype=q.dtype, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        blin.rope(q, grid=(2 ** 24, 1, 1), rope_split=(16, 24, 24))
    with pytest.raises(torch.OutOfMemoryError):
        blin.decay_prefill(q, q, q, torch.zeros(4096, device="cuda"))


@pytest.mark.gpu
def test_the_decayed_attention_refuses_what_autograd_would_record():
    q, k, v = (torch.randn(2, 3, 5, 64, device="cuda") for _ in range(3))
    lg, pool = torch.full((3,), -0.1, device="cuda"), torch.zeros(2, 3, 64, 64, device="cuda")
    one = [x[:, :, 0] for x in (q, k, v)]
    want, step = blin.decay_prefill(q, k, v, lg), blin.decay_step(*one, lg, pool.clone())
    for i in range(6):  # q, k, v, log_decay, the pool, out
        def leaf(j, t):
            return t.detach().clone().requires_grad_() if i == j else t
        full = [leaf(j, t) for j, t in enumerate((q, k, v, lg))]
        last = [leaf(j, t.contiguous()) for j, t in enumerate((*one, lg))]
        state, out, out1 = leaf(4, pool.clone()), leaf(5, torch.empty_like(q)), leaf(5, torch.empty_like(one[0]))
        with pytest.raises(RuntimeError, match="gradient"):
            blin.decay_prefill(*full, state=state, out=out)
        with pytest.raises(RuntimeError, match="gradient"):
            blin.decay_step(*last, state, out=out1)
        for off in (torch.no_grad(), torch.inference_mode()):
            with off:
                assert torch.equal(blin.decay_prefill(*full, state=state.clone(), out=out), want)
                assert torch.equal(blin.decay_step(*last, state.clone(), out=out1), step)


SPLIT, GRID = (16, 24, 16), (3, 4, 5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("given", [False, True])
def test_autograd_records_rope(dtype, inverse, given):
    """The gradient of a weighted sum of both outputs is the weights rotated back: to the bits, as it is the
    same kernel; that this is the formula's gradient and the differences' is test_rope's."""
    B, N, d = 2, 60, 64
    gen = torch.Generator(device="cuda").manual_seed(0)
    q, k, gq, gk = (torch.randn(B, h, N, d, generator=gen, device="cuda").to(dtype) for h in (3, 2, 3, 2))
    kw = dict(rope_split=SPLIT, theta=5e3)
    if given:
        kw["positions"] = torch.randint(-9, 9999, (B, N, 3), generator=gen, device="cuda", dtype=torch.int32)
    else:
        kw.update(grid=GRID, t0=2)
    want = blin.rope(q, k, inverse=inverse, **kw)
    back = blin.rope(gq, gk, inverse=not inverse, **kw)
    for need in ((True, True), (True, False), (False, True)):
        x, y = q.clone().requires_grad_(need[0]), k.clone().requires_grad_(need[1])
        outs = blin.rope(x, y, inverse=inverse, **kw)
        assert all(torch.equal(o, w) and o.requires_grad == n for o, w, n in zip(outs, want, need))
        torch.autograd.backward([o for o, n in zip(outs, need) if n], [g for g, n in zip((gq, gk), need) if n])
        for t, g, n in zip((x, y), back, need):
            assert torch.equal(t.grad, g) if n else t.grad is None
    # one output used, by a sum (a gradient without strides); q alone; a second derivative
    x, y = q.clone().requires_grad_(), k.clone().requires_grad_()
    a, b = blin.rope(x, y, inverse=inverse, **kw)
    b.sum().backward()
    assert x.grad is None and torch.equal(y.grad, blin.rope(torch.ones_like(k), inverse=not inverse, **kw))
    z = blin.rope(x, inverse=inverse, **kw)
    (g,) = torch.autograd.grad(z, x, gq.clone().requires_grad_(), create_graph=True)
    assert torch.equal(z, want[0]) and torch.equal(g, back[0]) and g.requires_grad
    u = gq.clone().requires_grad_()
    (g,) = torch.autograd.grad(z, x, u, create_graph=True)
    (g2,) = torch.autograd.grad(g, u, q)
    assert torch.equal(g2, want[0])


@pytest.mark.gpu
def test_rope_with_out_refuses_what_autograd_would_record():
    q, k = (torch.randn(1, 2, 60, 64, device="cuda") for _ in range(2))
    kw = dict(grid=GRID, rope_split=SPLIT)
    want = blin.rope(q, k, **kw)
    x = q.clone().requires_grad_()
    for args, out in (((x, k), (torch.empty_like(q), torch.empty_like(k))), ((x, k), (x, k)), ((k, x), (k, x)),
                      ((q, k), (torch.empty_like(q), torch.empty_like(q).requires_grad_()))):
        with pytest.raises(RuntimeError, match="gradient"):
            blin.rope(*args, out=out, **kw)
    assert torch.equal(x, q)
    with torch.no_grad():
        got = blin.rope(x, k.clone(), out=(x, torch.empty_like(k)), **kw)
        assert got[0] is x and torch.equal(x, want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_a_training_step_through_rope_in_a_graph():
    """Forward and backward captured and replayed: the eager gradients."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    w, x = (torch.randn(1, 2, 60, 64, generator=gen, device="cuda") for _ in range(2))

    def grads(x):
        q = (x * 2).requires_grad_()
        a, b = blin.rope(q, q * 0.5, grid=GRID, rope_split=SPLIT)
        return torch.autograd.grad((a * w).sum() + (b * b * w).sum(), q)[0]

    static = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads(static)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = grads(static)
    for seed in (2, 3):
        new = torch.randn(x.shape, generator=gen, device="cuda")
        static.copy_(new)
        g.replay()
        assert torch.equal(out, grads(new))


@pytest.mark.gpu
def test_autograd_learns_of_tensors_that_were_written_to():
    """A tensor saved for a backward pass and then overwritten is an error there, not a wrong gradient."""
    q, k, v = (torch.randn(2, 3, 60, 64, device="cuda") for _ in range(3))
    lg, pool = torch.full((3,), -0.1, device="cuda"), torch.zeros(2, 3, 64, 64, device="cuda")
    kw = dict(grid=GRID, rope_split=SPLIT)
    ws = torch.empty(blin.decay_workspace_size(2, 3, 60, 64, torch.float32), dtype=torch.uint8, device="cuda")

    def writes(call, *to):
        before = [t._version for t in to]
        read = [t._version for t in (k, v, lg)]
        call()
        assert [t._version for t in to] == [n + 1 for n in before] and [t._version for t in (k, v, lg)] == read

    o, o1, r = torch.empty_like(q), torch.empty_like(q[:, :, 0]), torch.empty_like(q)
    writes(lambda: blin.decay_prefill(q, k, v, lg, state=pool, out=o, workspace=ws), pool, o, ws)
    writes(lambda: blin.decay_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], lg, pool, out=o1), pool, o1)
    writes(lambda: blin.rope(q, k, out=(q, r), **kw), q, r)
    w = torch.ones_like(q, requires_grad=True)
    y = (w * q).sum()
    blin.rope(q, out=q, **kw)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    with torch.inference_mode():
        a, p = torch.zeros_like(q), torch.zeros_like(pool)
        blin.decay_prefill(q, k, v, lg, state=p, out=a)
    blin.decay_prefill(q, k, v, lg, state=p, out=a)  # tensors of inference mode count no versions


@pytest.mark.gpu
def test_inputs_live_until_the_calls_stream_has_read_them():
    """A call waits on a busy stream while its caller drops the inputs and the current stream writes to
    memory of their sizes: the call must still read the inputs."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    B, H, N, d = 2, 4, 4096, 64
    big = torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
    y = torch.empty_like(big)
    side = torch.cuda.Stream()
    q, k, v = (torch.randn(B, H, N, d, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
    lg, slots = torch.tensor([-0.1, -0.01, 0.0, -0.5], device="cuda"), torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([N, N - 77], dtype=torch.int32, device="cuda")
    pos = torch.randint(0, 9999, (B, N, 3), generator=gen, device="cuda", dtype=torch.int32)
    pool = torch.randn(3, H, d, d, generator=gen, device="cuda")
    need = blin.decay_workspace_size(B, H, N, d)
    one = [x[:, :, 3].contiguous() for x in (q, k, v)]

    def prefill(q, k, v, lg, slots, lengths, pool, ws, **kw):
        return blin.decay_prefill(q, k, v, lg, state=pool, slots=slots, lengths=lengths, workspace=ws, **kw)

    def step(q, k, v, lg, slots, pool, **kw):
        return blin.decay_step(q, k, v, lg, pool, slots=slots, **kw)

    def rope(q, k, pos, **kw):
        return torch.cat(blin.rope(q, k, positions=pos, rope_split=SPLIT, **kw)) if not kw else blin.rope(
            q, k, positions=pos, rope_split=SPLIT, **kw)

    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert need > 16
    for call, args in ((prefill, (q, k, v, lg, slots, lengths, pool, ws)), (step, (*one, lg, slots, pool)),
                       (rope, (q, k, pos))):
        want = call(*(t.clone() for t in args))
        for last in (False, True):  # first a run that loads every kernel, which may wait for the device
            copies = [t.clone() for t in args]
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                for _ in range(200):  # about a tenth of a second
                    torch.matmul(big, big, out=y)
            got = call(*copies, stream=side)
            del copies
            late = [torch.empty_like(t).view(torch.uint8).fill_(0xFF) for t in args for _ in range(8)]
            torch.cuda.current_stream().synchronize()
            assert not last or not side.query()  # the call had not begun when the memory was written to
            torch.cuda.synchronize()
            assert torch.equal(got if torch.is_tensor(got) else torch.cat(got), want)
            del late
