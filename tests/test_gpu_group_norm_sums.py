"""dweight and dbias over many rows, of many heads and of few."""
import numpy as np
import pytest

U32 = 2.0 ** -24


@pytest.mark.parametrize("B,H,N,d", [(1, 2048, 1 << 20, 64), (4, 65535, 1 << 16, 16), (2, 4096, 30000, 128), (1, 1, 1 << 20, 64)])
def test_no_slice_has_more_than_2048_rows(B, H, N, d):
    """The workspace has a row of sums for every slice."""
    from test_learned_neural_amd import titans_mem as tmm
    need = tmm.group_norm_backward_workspace_bytes(tmm.make_norm_desc(B, H, N, d))
    slices = need // (2 * 4 * H * d)
    assert slices * 2048 >= B * N
    assert slices <= max(512, -(-B * N // 2048))


@pytest.mark.parametrize("B,H,N", [(1 << 18, 1, 0x7fffffff), (1 << 10, 200, 0x7fffffff), (1, 65535, 0x7fffffff)])
def test_a_launch_stays_under_2_32_threads(B, H, N):
    from test_learned_neural_amd import titans_mem as tmm
    slices = tmm.group_norm_backward_workspace_bytes(tmm.make_norm_desc(B, H, N, 1)) // (2 * 4 * H)
    assert 0 < slices * H * 256 < 1 << 32


@pytest.mark.gpu
@pytest.mark.parametrize("H,N", [(2048, 1 << 19), (3000, 33333), (1, 1 << 20), (2, 300000)])
def test_sums_of_equal_terms(H, N):
    """Equal terms: every rounding of a running sum may fall to the same side.  A slice of up to 2048 rows leaves a
    thread 2048 / 16 terms (16 groups of one channel in a workgroup), 16 threads' sums and up to 2048 slices' in 16
    strands are joined: 128 + 16 + 128 + 16 additions, each off by u of the sum at most."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    x = torch.zeros(1, N, H, device="cuda")
    dout = torch.full((1, N, H), 1 / 3, device="cuda")
    g = tmm.group_norm_backward(x, None, None, dout, H=H, activation=tmm.ACT_NONE)
    want = float(dout[0, 0, 0].double()) * N
    off = (g["bias"].double() - want).abs().max().item() / want
    assert off <= 288 * U32, off / U32
    assert (g["weight"] == 0).all()
    out = tmm.group_norm(x, None, torch.arange(H, device="cuda", dtype=torch.float32), H=H, activation=tmm.ACT_NONE)
    assert (out == torch.arange(H, device="cuda")).all()
