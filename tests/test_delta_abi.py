"""Host-only checks of the delta memory's and the group norm's C entries: each
refusal is one defect in a call that is otherwise right, with device addresses
that are never dereferenced."""
import pytest

from test_learned_neural_amd import titans_mem as tmm

BASE = 0x7f0000000000


def _lay(sizes):
    at, cur = {}, BASE
    for name, n in sizes.items():
        at[name] = cur
        cur += (max(n, 16) + 4095) // 4096 * 4096 + 4096
    return at


class Delta:
    def __init__(self, io="bf16", N=100, **kw):
        self.desc = tmm.make_delta_desc(2, 6, 3, N, 64, io, **kw)
        e = 2 if io == "bf16" else 4
        self.ws = max(tmm.delta_workspace_bytes(self.desc), 16)
        self.p = _lay(dict(k=2 * 3 * N * 64 * e, v=2 * 6 * N * 64 * e, q=2 * 3 * N * 64 * e, alpha=2 * 6 * N * 4,
                           theta=2 * 6 * N * 4, lengths=8, W_in=12 * 64 * 64 * 4, y=2 * 6 * N * 64 * e,
                           W_out=12 * 64 * 64 * 4, ws=self.ws))

    def call(self, **over):
        p = {**self.p, "ws_bytes": self.ws, **over}
        return tmm.raw_delta_forward(self.desc, p["k"], p["v"], p["q"], p["alpha"], p["theta"], p["lengths"],
                                     p["W_in"], p["y"], p["W_out"], p["ws"], p["ws_bytes"], 0)


class Norm:
    def __init__(self, io="bf16", **kw):
        self.desc = tmm.make_norm_desc(2, 3, 50, 32, io, **kw)
        n = 2 * 50 * 96 * (2 if io == "bf16" else 4)
        self.ws = tmm.group_norm_backward_workspace_bytes(self.desc)
        self.p = _lay(dict(x=n, gate=n, weight=384, bias=384, lengths=8, out=n, dout=n, dx=n, dgate=n, dweight=384,
                           dbias=384, ws=max(self.ws, 16)))

    def call(self, **over):
        p = {**self.p, **over}
        return tmm.raw_group_norm(self.desc, p["x"], p["gate"], p["weight"], p["bias"], p["lengths"], p["out"], 0)

    def back(self, **over):
        p = {**self.p, "ws_bytes": self.ws, **over}
        return tmm.raw_group_norm_backward(self.desc, p["x"], p["gate"], p["weight"], p["bias"], p["lengths"], p["dout"],
                                           p["dx"], p["dgate"], p["dweight"], p["dbias"], p["ws"], p["ws_bytes"], 0)


@pytest.mark.parametrize("field,value,status", [
    ("abi_version", 2, "INVALID"), ("B", 0, "INVALID"), ("H", 0, "INVALID"), ("Hk", 0, "INVALID"),
    ("Hk", 4, "INVALID"), ("N", -1, "INVALID"), ("d", 0, "INVALID"), ("io_dtype", 2, "INVALID"),
    ("flags", tmm.FLAG_CHUNK_GATES, "INVALID"), ("d", 129, "UNSUPPORTED"), ("B", 1 << 30, "UNSUPPORTED"),
    ("N", 0x7fffffff, None)])
def test_delta_descriptor(field, value, status):
    c = Delta()
    setattr(c.desc, field, value)
    want = 0 if status is None else getattr(tmm, "ERR_" + status)
    got = tmm.delta_workspace_bytes(c.desc)
    assert got >= 0 if status is None else got == want
    path = tmm.delta_select_path(c.desc)
    assert path in (tmm.PATH_DELTA_RECURRENT, tmm.PATH_DELTA_CHUNKED) if status is None else path == want
    if status is not None:
        assert c.call() == want


@pytest.mark.parametrize("name", ["k", "v", "q", "alpha", "theta", "W_in", "y", "W_out"])
def test_delta_pointers(name):
    c = Delta()
    assert c.call(**{name: 0}) == tmm.ERR_INVALID
    assert c.call(**{name: c.p[name] + 8}) == tmm.ERR_INVALID


def test_delta_optional_pointers_are_checked_for_alignment():
    c = Delta()
    assert c.call(lengths=c.p["lengths"] + 4) == tmm.ERR_INVALID
    assert c.call(ws=c.p["ws"] + 4) == tmm.ERR_INVALID


@pytest.mark.parametrize("out", ["y", "W_out"])
@pytest.mark.parametrize("other", ["k", "v", "q", "alpha", "theta", "lengths", "W_in", "y", "W_out"])
def test_delta_overlaps(out, other):
    if out == other:
        return
    c = Delta()
    assert c.call(**{out: c.p[other] + (16 if {out, other} == {"W_out", "W_in"} else 0)}) == tmm.ERR_ALIAS


def test_delta_small_workspace_is_refused():
    c = Delta(N=20000)      # few streams and many tokens: cut into segments, which need one
    assert tmm.delta_workspace_bytes(c.desc) == c.ws > 0
    assert c.call(ws_bytes=c.ws - 1) == tmm.ERR_WORKSPACE
    assert c.call(ws=0) == tmm.ERR_WORKSPACE
    assert c.call(ws=c.p["v"]) == tmm.ERR_ALIAS
    assert tmm.delta_workspace_bytes(Delta(N=100).desc) == 0


@pytest.mark.parametrize("field,value,status", [
    ("abi_version", 0, "INVALID"), ("B", 0, "INVALID"), ("H", -1, "INVALID"), ("N", -1, "INVALID"), ("d", 0, "INVALID"),
    ("io_dtype", 9, "INVALID"), ("activation", 2, "INVALID"), ("eps", -1.0, "INVALID"), ("eps", float("nan"), "INVALID"),
    ("eps", float("inf"), "INVALID"), ("flags", 1, "INVALID"), ("d", 1025, "UNSUPPORTED"), ("H", 65536, "UNSUPPORTED")])
def test_norm_descriptor(field, value, status):
    c = Norm()
    setattr(c.desc, field, value)
    want = getattr(tmm, "ERR_" + status)
    assert c.call() == want and c.back() == want
    assert tmm.group_norm_backward_workspace_bytes(c.desc) == want


def test_norm_pointers_and_overlaps():
    c = Norm()
    for name in ("x", "out"):
        assert c.call(**{name: 0}) == tmm.ERR_INVALID
    for name in ("x", "out", "gate", "weight", "bias", "lengths"):
        assert c.call(**{name: c.p[name] + 8}) == tmm.ERR_INVALID
    for name in ("x", "gate", "weight", "bias", "lengths"):
        assert c.call(out=c.p[name]) == tmm.ERR_ALIAS
    for name in ("x", "dout", "dx", "dweight", "dbias", "dgate", "gate"):
        assert c.back(**{name: 0}) == tmm.ERR_INVALID, name
    for name in ("x", "gate", "weight", "bias", "lengths", "dout", "dx", "dgate", "dweight", "dbias", "ws"):
        assert c.back(**{name: c.p[name] + 4}) == tmm.ERR_INVALID, name
    for out in ("dx", "dgate", "dweight", "dbias", "ws"):
        for name in ("x", "gate", "weight", "bias", "lengths", "dout", "dx", "dgate", "dweight", "dbias"):
            if name != out:
                assert c.back(**{out: c.p[name]}) == tmm.ERR_ALIAS, (out, name)
    assert c.back(ws=0) == tmm.ERR_WORKSPACE
    assert c.back(ws_bytes=c.ws - 1) == tmm.ERR_WORKSPACE


def test_wrappers_refuse_before_the_library():
    import torch
    B, H, Hk, N, d = 1, 2, 1, 3, 8
    a = dict(k=torch.zeros(B, Hk, N, d), v=torch.zeros(B, H, N, d), q=torch.zeros(B, Hk, N, d),
             alpha=torch.zeros(B, H, N), theta=torch.zeros(B, H, N), W_in=torch.zeros(B, H, d, d))

    def call(**over):
        x = {**a, **over}
        lengths = x.pop("lengths", None)
        return tmm.delta_forward(*x.values(), lengths=lengths)

    for over in (dict(q=torch.zeros(B, Hk, N, d + 1)), dict(v=torch.zeros(B, H, N, d, dtype=torch.bfloat16)),
                 dict(alpha=torch.zeros(B, H, N, dtype=torch.float64)), dict(k=torch.zeros(B, Hk, d, N).transpose(2, 3)),
                 dict(lengths=torch.zeros(B, dtype=torch.int64)), dict(W_in=torch.zeros(B, H, d * d)),
                 dict(k=torch.zeros(Hk, N, d)), {}):     # the last: right, but on the CPU
        with pytest.raises(ValueError):
            call(**over)
    x = torch.zeros(2, 3, 4, 8)
    for args, kw in (((x.half(),), {}), ((x,), dict(H=2)), ((x[0],), {}), ((x[0],), dict(H=3)),
                     ((x, torch.zeros(23)), {}), ((x,), dict(gate=torch.zeros(2, 4, 24, dtype=torch.bfloat16))), ((x,), {})):
        with pytest.raises(ValueError):
            tmm.group_norm(*args, **kw)
    with pytest.raises(ValueError):
        tmm.group_norm_backward(x, None, None, torch.zeros(2, 4, 23))


class DeltaGrad(Delta):
    def __init__(self, io="bf16", N=100, **kw):
        super().__init__(io, N, **kw)
        e = 2 if io == "bf16" else 4
        key, val, gate, state = 2 * 3 * N * 64 * e, 2 * 6 * N * 64 * e, 2 * 6 * N * 4, 12 * 64 * 64 * 4
        self.ws = tmm.delta_backward_workspace_bytes(self.desc)
        self.p = _lay(dict(k=key, v=val, q=key, alpha=gate, theta=gate, lengths=8, W_in=state, dy=val, dW_out=state,
                           dk=key, dv=val, dq=key, dalpha=gate, dtheta=gate, dW_in=state, ws=self.ws))

    def call(self, **over):
        p = {**self.p, "ws_bytes": self.ws, **over}
        return tmm.raw_delta_backward(self.desc, *(p[n] for n in (
            "k", "v", "q", "alpha", "theta", "lengths", "W_in", "dy", "dW_out", "dk", "dv", "dq", "dalpha", "dtheta",
            "dW_in", "ws", "ws_bytes")), 0)


@pytest.mark.parametrize("field,value,status", [
    ("abi_version", 2, "INVALID"), ("H", 7, "INVALID"), ("N", -2, "INVALID"), ("io_dtype", -1, "INVALID"),
    ("d", 200, "UNSUPPORTED"), ("B", 1 << 23, "UNSUPPORTED")])
def test_delta_backward_descriptor(field, value, status):
    c = DeltaGrad()
    setattr(c.desc, field, value)
    want = getattr(tmm, "ERR_" + status)
    assert tmm.delta_backward_workspace_bytes(c.desc) == want and c.call() == want


def test_delta_backward_pointers_and_overlaps():
    c = DeltaGrad()
    names = [n for n in c.p if n != "ws"]
    for name in names:
        assert c.call(**{name: c.p[name] + 8}) == tmm.ERR_INVALID, name
        if name not in ("lengths", "dW_out"):
            assert c.call(**{name: 0}) == tmm.ERR_INVALID, name
    for out in ("dk", "dv", "dq", "dalpha", "dtheta", "dW_in", "ws"):
        for name in names:
            if name != out:
                assert c.call(**{out: c.p[name]}) == tmm.ERR_ALIAS, (out, name)
    assert c.call(ws=0) == tmm.ERR_WORKSPACE
    assert c.call(ws_bytes=c.ws - 1) == tmm.ERR_WORKSPACE


def test_delta_limits_of_a_launch():
    """A launch has fewer than 2^32 threads: streams up to 2^20, a gradient's chunks times 256 (512 past d = 64)."""
    def desc(B=1, H=1, N=64, d=16):
        return tmm.make_delta_desc(B, H, H, N, d)

    for N in (4, 64):
        assert tmm.delta_select_path(desc(B=1 << 19, H=2, N=N)) >= 0
        assert tmm.delta_select_path(desc(B=1 << 19, H=2 + 1, N=N)) == tmm.ERR_UNSUPPORTED
    for d, threads in ((64, 256), (65, 512)):
        chunks = (1 << 32) // threads
        ld = (d + 15) // 16 * 16
        fits = desc(N=32 * (chunks - 1), d=d)
        assert tmm.delta_backward_workspace_bytes(fits) == (chunks - 1) * 8 * (ld * ld + 32 * ld)
        assert tmm.delta_backward_workspace_bytes(desc(N=32 * chunks, d=d)) == tmm.ERR_UNSUPPORTED
        assert tmm.delta_backward_workspace_bytes(desc(B=2, N=16 * chunks, d=d)) == tmm.ERR_UNSUPPORTED


def test_delta_longest_sequence_is_cut_as_others_are():
    longest, long = (tmm.delta_workspace_bytes(tmm.make_delta_desc(1, 1, 1, N, 64)) for N in (0x7fffffff, 1 << 30))
    assert longest == long > 0
    assert tmm.delta_backward_workspace_bytes(tmm.make_delta_desc(1, 1, 1, 0x7fffffff, 64)) == tmm.ERR_UNSUPPORTED


def test_dimensions_past_32_bits_do_not_wrap():
    """A tensor can have 2^32 tokens; the descriptors' fields cannot hold that many."""
    import torch
    big = 1 << 32
    for keys, vals in (((1, 1, big, 1), (1, 1, big, 1)), ((big + 1, 1, 4, 4), (big + 1, 1, 4, 4)),
                       ((1, 1, 4, 4), (1, big + 1, 4, 4))):
        with pytest.raises(ValueError, match="2\\^31"):
            tmm._DeltaPlan(keys, vals, torch.bfloat16, 0)
    for shape, H in (((1, 1, big, 1), None), ((big + 1, 4, 8), 2), ((1, 4, big * 8), 2)):
        with pytest.raises(ValueError, match="2\\^31"):
            tmm._NormPlan(shape, torch.float32, H, tmm.ACT_SILU, 1e-5)


def test_a_query_before_torch_is_imported_leaves_one_hip_runtime():
    """torch brings a HIP runtime of its own: with two in a process no launch on torch's tensors works."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("from test_learned_neural_amd import titans_mem as t\n"
            "t.delta_workspace_bytes(t.make_delta_desc(1, 1, 1, 64, 64))\n"
            "import torch\n"
            "files = {l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}\n"
            "assert len(files) == 1, files\n")
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True, timeout=300)
