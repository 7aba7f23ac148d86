"""Workspaces of exactly the bytes asked for, with a border behind them that has to stay: the attention's gradient,
the step and the projection's gradient, at sizes whose pieces end at odd places.  Results are those of a new workspace."""
import pytest

pytestmark = pytest.mark.gpu


def _tight(need):
    """(uint8 [need] at 16 bytes, whether the border behind it is whole)."""
    import torch
    buf = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    return buf[:need], lambda: bool((buf[need:] == 0x5a).all())


def _rand(seed, ty, *shapes):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").to(ty) for s in shapes]


def _type(io):
    import torch
    return torch.bfloat16 if io == "bf16" else torch.float32


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk,N,d", [(1, 1, 1, 1), (3, 1, 333, 33), (5, 5, 1001, 64), (8, 2, 700, 7), (2, 2, 129, 128)])
@pytest.mark.parametrize("packed", [False, True])
def test_attention_gradient(H, Hk, N, d, io, packed):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    lead = () if packed else (1,)
    q, k, v, do = _rand(1, _type(io), lead + ((N, H, d) if packed else (H, N, d)), *[lead + ((N, Hk, d) if packed else (Hk, N, d))] * 2,
                        lead + (N, H * d))
    kw = dict(offsets=torch.tensor([0, N // 3, N], dtype=torch.int32, device="cuda")) if packed else {}
    out, lse = tmm.attention(q, k, v, **kw)
    need = tmm.attention_backward_workspace_bytes(tmm.make_attention_desc(
        2 if packed else 1, H, Hk, N, d, io, flags=tmm.FLAG_CHANNELS_LAST if packed else 0), packed)
    ws, whole = _tight(need)
    want, got = tmm.attention_backward(q, k, v, out, lse, do, **kw), tmm.attention_backward(q, k, v, out, lse, do, workspace=ws, **kw)
    assert all(torch.equal(want[n], got[n]) for n in "qkv") and whole()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,n,C,d", [(1, 1, 1, 800, 33), (1, 3, 1, 5000, 1), (3, 1, 5, 900, 7), (1, 2, 3, 9001, 128)])
def test_step(B, H, n, C, d, io):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    q, k, v = _rand(2, _type(io), (B, H, n, d), *[(B, H, C, d)] * 2)
    ln = torch.full((B,), C, dtype=torch.int32, device="cuda")
    ws, whole = _tight(tmm.attention_step_workspace_bytes(tmm.make_attention_step_desc(B, H, H, n, C, d, io)))
    assert ws.numel() > 0
    assert torch.equal(tmm.attention_step(q, k, v, ln), tmm.attention_step(q, k, v, ln, workspace=ws)) and whole()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("M,K,O", [(1, 1, 1), (3, 5, 7), (1001, 33, 77), (5000, 64, 129), (4096, 256, 512), (0, 8, 9)])
def test_projection_gradient(M, K, O, io, act):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    x, w, do, pre = _rand(3, _type(io), (M, K), (O, K), (M, O), (M, O))
    a = tmm.ACT_SILU if act else tmm.ACT_NONE
    kw = dict(pre=pre if act else None, activation=a)
    ws, whole = _tight(tmm.projection_backward_workspace_bytes(tmm.make_projection_desc(M, K, O, io, a)))
    want, got = tmm.projection_backward(x, w, do, **kw), tmm.projection_backward(x, w, do, workspace=ws, **kw)
    assert all(torch.equal(want[n], got[n]) for n in want) and whole()
