"""The projection and its gradient against the fp64 oracle.

Bounds, element by element (u = 2^-24, h = 2^-8 for a bf16 result, else 0): a
sum of n products, each off by at most 4 u (fp32 planes; bf16 products are
exact) and summed in fp32 with independent roundings, by 8 u sqrt(n) sum |terms|.
SiLU's slope is below 1.1, its value off by 8 u |z| more (16 u of the slope's
terms in dz).  out ends in h + u of itself and of the residual's sum.  A bf16 dz
is off by h for dx, and by 2^-16 as the two numbers that dweight takes.
"""
import numpy as np
import pytest

from attention_util import H16, U, dtype, near, rounded
from oracle import attention_oracle as ao

pytestmark = pytest.mark.gpu

#          rows  K     O    io
SHAPES = [(1, 64, 64, "bf16"), (1, 1, 1, "f32"), (1, 1, 1, "bf16"), (3, 7, 5, "bf16"), (16, 100, 30, "f32"),
          (17, 33, 65, "bf16"), (64, 1000, 24, "bf16"), (64, 256, 40, "f32"), (65, 256, 40, "f32"), (65, 8, 8, "bf16"),
          (100, 31, 129, "f32"), (130, 72, 200, "bf16"), (257, 65, 66, "bf16"), (300, 500, 77, "f32"), (300, 500, 76, "f32"),
          (700, 96, 1000, "bf16"), (2000, 130, 64, "bf16"), (3001, 40, 136, "f32"), (9000, 64, 1000, "f32"),
          (13000, 40, 520, "bf16"), (50000, 24, 264, "bf16"), (132000, 40, 264, "bf16"), (33100, 8, 1032, "bf16")]


def _draw(seed, M, K, O, io):
    rng = np.random.default_rng([seed, M, K, O])
    t, f = {}, {}
    for name, x in (("x", rng.standard_normal((M, K))), ("weight", rng.standard_normal((O, K)) / np.sqrt(K)),
                    ("residual", rng.standard_normal((M, O))), ("dout", rng.standard_normal((M, O)))):
        a, f[name] = rounded(x, io)
        t[name] = a.cuda()
    a, f["bias"] = rounded(0.3 * rng.standard_normal(O), "f32")
    t["bias"] = a.cuda()
    return t, f


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_gradient(shape, silu):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    M, K, O, io = shape
    t, f = _draw(31, M, K, O, io)
    h = H16 if io == "bf16" else 0.0
    act = tmm.ACT_SILU if silu else tmm.ACT_NONE
    pre = torch.empty(M, O, dtype=dtype(io), device="cuda")
    out = tmm.projection(t["x"], t["weight"], t["bias"], residual=t["residual"], activation=act, pre_out=pre)
    want, z = ao.projection(f["x"], f["weight"], f["bias"], f["residual"], silu)
    ez = 8 * U * np.sqrt(K) * (np.abs(f["x"]) @ np.abs(f["weight"]).T) + 4 * U * (np.abs(z) + np.abs(f["bias"]))
    near("pre", pre, z, ez + (h + U) * np.abs(z))
    near("out", out, want, 1.1 * ez + 8 * U * np.abs(z) + (h + 2 * U) * (np.abs(want) + 2 * U * np.abs(f["residual"])) +
         2 * U * np.abs(f["residual"]))
    # without bias and residual, and in place over the residual
    plain = tmm.projection(t["x"], t["weight"])
    w0, _ = ao.projection(f["x"], f["weight"])
    near("plain", plain, w0, ez + (h + U) * np.abs(w0))
    again = t["residual"].clone()
    assert tmm.projection(t["x"], t["weight"], t["bias"], residual=again, activation=act, out=again) is again
    assert torch.equal(again, out)
    # the gradient, at the stored z
    zd = pre.double().cpu().numpy() if silu else None
    got = tmm.projection_backward(t["x"], t["weight"], t["dout"], pre=pre if silu else None, activation=act)
    dx, dw, db = ao.projection_backward(f["x"], f["weight"], f["dout"], zd)
    dz = np.abs(f["dout"] if zd is None else f["dout"] * ao.silu_slope(zd))
    edz = 0 if zd is None else 16 * U * np.abs(f["dout"]) * (1 + np.abs(zd) / 4)
    near("dx", got["x"], dx, (8 * U * np.sqrt(O) * dz + edz + (h * dz if silu else 0)) @ np.abs(f["weight"]) +
         (h + U) * np.abs(dx))
    two = (2.0 ** -16 if silu and io == "bf16" else 0) * dz + edz
    near("dweight", got["weight"], dw, (8 * U * np.sqrt(M) * dz + two).T @ np.abs(f["x"]) + 1e-30)
    near("dbias", got["bias"], db, (8 * U * np.sqrt(M) * dz + edz).sum(0) + 1e-30)
    assert all(torch.equal(got[n], x) for n, x in tmm.projection_backward(
        t["x"], t["weight"], t["dout"], pre=pre if silu else None, activation=act).items())


# rows that are not made of 16-byte pieces: fewer elements than a piece has, pieces
# that pass a row's end by each number of elements, large tiles and small ones
ODD = [(65, 3, 2, "f32"), (70, 5, 3, "f32"), (90, 2, 3, "bf16"), (90, 9, 7, "bf16"), (66, 66, 67, "f32"), (130, 129, 63, "f32"),
       (200, 63, 131, "f32"), (100, 17, 130, "bf16"), (100, 18, 131, "bf16"), (100, 19, 132, "bf16"), (100, 20, 133, "bf16"),
       (100, 21, 134, "bf16"), (100, 22, 135, "bf16"), (100, 23, 129, "bf16"), (5000, 43, 1001, "f32"), (9000, 43, 1001, "bf16"),
       (4100, 321, 333, "f32")]


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("shape", ODD, ids=str)
def test_rows_of_any_size(shape, silu):
    test_forward_and_gradient(shape, silu)


def test_rows_shapes_and_nothing_to_do():
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    x, w = torch.randn(2, 3, 5, 16, device="cuda"), torch.randn(8, 16, device="cuda")
    out = tmm.projection(x, w)
    assert out.shape == (2, 3, 5, 8) and torch.equal(out.reshape(30, 8), tmm.projection(x.reshape(30, 16), w))
    g = tmm.projection_backward(x, w, out)
    assert g["x"].shape == x.shape and g["weight"].shape == w.shape
    assert tmm.projection(x[0, 0, 0], w).shape == (8,)
    e = torch.empty(0, 16, device="cuda")
    assert tmm.projection(e, w).shape == (0, 8)
    for io, act in ((torch.float32, tmm.ACT_NONE), (torch.bfloat16, tmm.ACT_SILU)):
        z = torch.empty(0, 8, device="cuda", dtype=io)
        g = tmm.projection_backward(e.to(io), w.to(io), z, pre=z if act == tmm.ACT_SILU else None, activation=act)
        assert (g["weight"] == 0).all() and (g["bias"] == 0).all() and g["x"].shape == (0, 16)


@pytest.mark.parametrize("rows", [5, 200, 140000])
def test_a_nan_stays_in_its_row_and_column(rows):
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    for io in (torch.bfloat16, torch.float32):
        x, w = torch.randn(rows, 40, device="cuda").to(io), torch.randn(264, 40, device="cuda").to(io)
        want = tmm.projection(x, w)
        x[rows // 2, 39] = float("nan")
        w[200, 0] = float("inf")
        bad = torch.zeros(rows, 264, dtype=torch.bool, device="cuda")
        bad[rows // 2], bad[:, 200] = True, True
        got = tmm.projection(x, w)
        assert torch.equal(torch.isfinite(got), ~bad) and torch.equal(got[~bad], want[~bad])


def test_streams_and_graphs():
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    for rows in (3, 500, 140000):
        t, _ = _draw(32, rows, 64, 264, "bf16")

        def run():
            pre = torch.empty(rows, 264, device="cuda", dtype=torch.bfloat16)
            o = tmm.projection(t["x"], t["weight"], t["bias"], residual=t["residual"], activation=tmm.ACT_SILU, pre_out=pre)
            g = tmm.projection_backward(t["x"], t["weight"], t["dout"], pre=pre, activation=tmm.ACT_SILU)
            return [o, g["x"], g["weight"], g["bias"]]

        want = run()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = run()
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        for turn in range(3):
            t["x"].copy_(torch.randn_like(t["x"]))
            graph.replay()
            want = run()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (rows, turn)


def test_rows_past_32_bits():
    """More than 2^31 elements of x and out: the last rows are the same as alone."""
    import torch
    from test_learned_neural_amd import titans_mem as tmm
    rows = (1 << 22) + 100
    x = torch.zeros(rows, 520, device="cuda", dtype=torch.bfloat16)
    x[-300:] = torch.randn(300, 520, device="cuda").bfloat16()
    w = torch.randn(520, 520, device="cuda").bfloat16()
    out = tmm.projection(x, w)
    want = x[-300:].double() @ w.double().t()
    bound = 8 * U * 520 ** 0.5 * (x[-300:].double().abs() @ w.double().abs().t()) + (H16 + U) * want.abs()
    assert ((out[-300:].double() - want).abs() <= bound).all() and (out[:-300] == 0).all()
    g = tmm.projection_backward(x, w, out)
    near("dx", g["x"][-300:], (out[-300:].double() @ w.double()).cpu().numpy(),
         (8 * U * 520 ** 0.5 * (out[-300:].double().abs() @ w.double().abs()) + (H16 + U) * (
             out[-300:].double() @ w.double()).abs()).cpu().numpy())
    ref = out[-300:].double().t() @ x[-300:].double()
    size = out[-300:].double().abs().t() @ x[-300:].double().abs()
    assert ((g["weight"].double() - ref).abs() <= 8 * U * 300 ** 0.5 * size).all()
