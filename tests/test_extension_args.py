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
