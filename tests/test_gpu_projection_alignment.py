"""The projection's buffers at every multiple of 16 bytes that no larger power of two divides."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,O", [(5, 64, 64), (200, 64, 72), (1800, 64, 1800), (33000, 64, 1032)])
def test_at_16_bytes(M, K, O, io):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    ty = torch.bfloat16 if io == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(71)

    def odd(t):
        by = 16 // t.element_size()
        at = torch.empty(t.numel() + 2 * by, dtype=t.dtype, device="cuda")[by:by + t.numel()].view(t.shape)
        assert at.data_ptr() % 32 == 16
        return at.copy_(t)

    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w, res, b, dout = r(M, K).to(ty), r(O, K).to(ty), r(M, O).to(ty), r(O), r(M, O).to(ty)
    pre = torch.empty_like(res)
    want = tmm.projection(x, w, b, residual=res, activation=tmm.ACT_SILU, pre_out=pre)
    back = tmm.projection_backward(x, w, dout, pre=pre, activation=tmm.ACT_SILU)
    xo, wo, bo, ro, po, do, to = (odd(t) for t in (x, w, b, res, torch.zeros_like(res), dout, torch.zeros_like(res)))
    tmm.projection(xo, wo, bo, residual=ro, activation=tmm.ACT_SILU, pre_out=po, out=to)
    assert torch.equal(to, want) and torch.equal(po, pre)
    tmm.projection(xo, wo, bo, residual=ro, activation=tmm.ACT_SILU, out=ro)      # in place
    assert torch.equal(ro, want)
    got = tmm.projection_backward(xo, wo, do, pre=po, activation=tmm.ACT_SILU)
    assert all(torch.equal(got[n], back[n]) for n in back)
