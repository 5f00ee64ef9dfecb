"""Host-side tests of what the calls of a serving step refuse (before any CUDA
call: they run on a machine without a GPU)."""
import ctypes

import pytest

from test_attn_host import INVALID, nv, step  # noqa: F401  (nv: the module's fixture)

MB = 1 << 20
APART = dict(requests=4, tokens=64, q_len=MB, ctx_len=2 * MB, cu_q=3 * MB, kv_len=4 * MB, pos=5 * MB, slot=6 * MB,
             block_table=7 * MB, schedule=8 * MB, cursor=9 * MB, cursor_out=10 * MB)


@pytest.mark.parametrize("bad", [dict(ctx_len=4 * MB), dict(q_len=4 * MB + 12), dict(ctx_len=3 * MB + 16),
                                 dict(q_len=3 * MB - 12), dict(ctx_len=5 * MB + 252), dict(q_len=6 * MB),
                                 dict(ctx_len=10 * MB - 12)])
def test_lengths_that_are_outputs_are_refused(nv, bad):
    assert nv.lib().nvfp4_attn_plan(step(nv, **{**APART, **bad}), None) == INVALID


@pytest.mark.parametrize("good", [{}, dict(cursor=10 * MB), dict(ctx_len=4 * MB + 16), dict(q_len=3 * MB + 20),
                                  dict(q_len=2 * MB), dict(ctx_len=5 * MB + 256)])
def test_lengths_beside_the_outputs_are_not(nv, good):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are not memory")
    assert nv.lib().nvfp4_attn_plan(step(nv, **{**APART, **good}), None) != INVALID


def test_zero_padding_fits_the_old_struct(nv):
    """The flag lies in what was padding at the struct's end."""
    assert ctypes.sizeof(nv._AttnIOC) == 72 and nv._AttnIOC.zero_padding.offset == 68
