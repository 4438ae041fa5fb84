"""A dispatch holds fewer than 2^32 work-items: of 256 threads each, 2^24
workgroups are one too many, and a call that needs them is refused by its size
before anything is enqueued."""
import segmented_gather_gemm_sgmv_amd as sg

P = [0x100000 * (i + 1) for i in range(8)]   # fake addresses, never dereferenced
SHAPE = -2


def test_the_gradient_of_2_to_the_24_tokens():
    """A workgroup per token."""
    T = 1 << 24
    assert sg.lib.sgmv_combine_rows_grad(P[0], 8, P[1], P[2], 8, P[3], 8, 90, P[4], P[5], T, 1, 8, 0, None) == SHAPE


def test_rows_of_a_workgroup_each():
    """264 columns of bf16 are 33 pieces of 16 bytes, more than share a wave: a workgroup per token."""
    T, d = 1 << 24, 264
    assert sg.lib.sgmv_spread_rows(P[0], d, 90, P[1], d, P[2], T, 1, d, 1, None) == SHAPE
    assert sg.lib.sgmv_combine_rows(P[0], d, None, 0, P[1], d, 90, P[2], None, T, 1, d, 1, None) == SHAPE


def test_rotary_write():
    """A workgroup per token of up to 256 pieces."""
    T = 1 << 24
    assert sg.lib.sgmv_rope_append(P[0], 128, P[1], 128, 1, None, 0, None, 0, None, None, 0, 0, 16, 128, P[2], None, T, P[3], 64,
                                   128, 0, 1, None) == SHAPE
