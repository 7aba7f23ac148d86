"""Host-only checks of the attention's and the projection's C entries: each
refusal is one defect in a call that is otherwise right, with device addresses
that are never dereferenced."""
import ctypes

import pytest

from test_learned_neural_amd import titans_mem as tmm

BASE = 0x7f0000000000


def _lay(sizes):
    at, cur = {}, BASE
    for name, n in sizes.items():
        at[name] = cur
        cur += (max(n, 16) + 4095) // 4096 * 4096 + 4096
    return at


class Call:
    def call(self, **over):
        p = {**self.p, "ws_bytes": getattr(self, "ws", 0), **over}
        return self.raw(self.desc, *(p[n] for n in self.names), 0)


class Attention(Call):
    raw = staticmethod(tmm.raw_attention)
    names = ("q", "k", "v", "offsets", "lengths", "out", "lse")

    def __init__(self, packed=False, **kw):
        self.desc = tmm.make_attention_desc(3, 6, 2, 100, 64, **kw)
        rows = (1 if packed else 3) * 100
        q, k = rows * 6 * 64 * 2, rows * 2 * 64 * 2
        self.p = _lay(dict(q=q, k=k, v=k, offsets=16, lengths=12, out=q, lse=rows * 6 * 4, dout=q, dq=q, dk=k, dv=k))
        self.p["lengths" if packed else "offsets"] = 0


class Backward(Attention):
    raw = staticmethod(tmm.raw_attention_backward)
    names = ("q", "k", "v", "offsets", "lengths", "out", "lse", "dout", "dq", "dk", "dv", "ws", "ws_bytes")

    def __init__(self, packed=False, **kw):
        super().__init__(packed, **kw)
        self.ws = tmm.attention_backward_workspace_bytes(self.desc, packed)
        self.p["ws"] = BASE + (1 << 32)


class Step(Call):
    raw = staticmethod(tmm.raw_attention_step)
    names = ("q", "k", "v", "k_new", "v_new", "lengths", "out", "ws", "ws_bytes")

    def __init__(self, C=4096, **kw):
        self.desc = tmm.make_attention_step_desc(3, 6, 2, 2, C, 64, **kw)
        q, k, n = 3 * 6 * 2 * 64 * 2, 3 * 2 * C * 64 * 2, 3 * 2 * 2 * 64 * 2
        self.ws = tmm.attention_step_workspace_bytes(self.desc)
        self.p = _lay(dict(q=q, k=k, v=k, k_new=n, v_new=n, lengths=12, out=q, ws=self.ws))


class Projection(Call):
    raw = staticmethod(tmm.raw_projection)
    names = ("x", "weight", "bias", "residual", "out", "pre")

    def __init__(self, **kw):
        self.desc = tmm.make_projection_desc(50, 64, 96, **kw)
        x, w, o = 50 * 64 * 2, 64 * 96 * 2, 50 * 96 * 2
        self.p = _lay(dict(x=x, weight=w, bias=384, residual=o, out=o, pre=o, dout=o, dx=x, dweight=2 * w, dbias=384))


class ProjectionBackward(Projection):
    raw = staticmethod(tmm.raw_projection_backward)
    names = ("x", "weight", "pre", "dout", "dx", "dweight", "dbias", "ws", "ws_bytes")

    def __init__(self, **kw):
        super().__init__(activation=tmm.ACT_SILU, **kw)
        self.ws = tmm.projection_backward_workspace_bytes(self.desc)
        self.p["ws"] = BASE + (1 << 32)


@pytest.mark.parametrize("kind", [Attention, Backward])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("field,value,status", [
    ("abi_version", 2, "INVALID"), ("B", 0, "INVALID"), ("H", 0, "INVALID"), ("Hk", 0, "INVALID"), ("Hk", 4, "INVALID"),
    ("N", -1, "INVALID"), ("d", 0, "INVALID"), ("io_dtype", 2, "INVALID"), ("window", -1, "INVALID"),
    ("prefix", -1, "INVALID"), ("scale", 0.0, "INVALID"), ("scale", -1.0, "INVALID"), ("scale", float("nan"), "INVALID"),
    ("scale", float("inf"), "INVALID"), ("flags", 1, "INVALID"), ("d", 129, "UNSUPPORTED"), ("H", 1 << 17, "UNSUPPORTED")])
def test_attention_descriptor(kind, packed, field, value, status):
    c = kind(packed)
    setattr(c.desc, field, value)
    if field == "H" and value > 100:
        c.desc.Hk = value
    assert c.call() == getattr(tmm, "ERR_" + status)
    assert tmm.attention_backward_workspace_bytes(c.desc, packed) == getattr(tmm, "ERR_" + status)


@pytest.mark.parametrize("packed", [False, True])
def test_attention_pointers(packed):
    for c, must, outs in ((Attention(packed), ("q", "k", "v", "out"), ("out", "lse")),
                          (Backward(packed), ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv"), ("dq", "dk", "dv", "ws"))):
        given = [n for n in c.names if n != "ws_bytes" and c.p[n]]
        for name in given:
            assert c.call(**{name: c.p[name] + 8}) == tmm.ERR_INVALID, name
        for name in must:
            assert c.call(**{name: 0}) == tmm.ERR_INVALID, name
        for out in outs:
            for name in given:
                if name != out:
                    assert c.call(**{out: c.p[name]}) == tmm.ERR_ALIAS, (out, name)
        assert c.call(offsets=c.p["q"] + (1 << 36), lengths=c.p["q"] + (1 << 37)) == tmm.ERR_INVALID   # not both
    c = Backward(packed)
    assert c.call(ws=0) == tmm.ERR_WORKSPACE and c.call(ws_bytes=c.ws - 1) == tmm.ERR_WORKSPACE


def test_attention_limits():
    """Launches stay under 2^24 workgroups of 256, distances within a tile under 2^32 bytes."""
    ok = lambda *a, **kw: tmm.attention_backward_workspace_bytes(tmm.make_attention_desc(*a, **kw))  # noqa: E731
    assert ok(1, 1, 1, 0x7fffffff, 64) == tmm.ERR_UNSUPPORTED
    assert ok(1, 1, 1, 1 << 28, 64) >= 0 and ok(1 << 20, 8, 8, 64, 64) == tmm.ERR_UNSUPPORTED
    assert ok(1, 1 << 15, 1 << 15, 32, 128) >= 0 and ok(1, (1 << 15) + 1, 1, 32, 128) == tmm.ERR_UNSUPPORTED
    assert ok(2, 4, 4, 0, 64) == 0
    c = Attention()
    c.desc.N = 0
    assert c.call() == tmm.OK
    assert ok(2, 4, 4, 5, 64, window=0x7fffffff, prefix=0x7fffffff) > 0


@pytest.mark.parametrize("field,value,status", [
    ("abi_version", 2, "INVALID"), ("B", 0, "INVALID"), ("H", 0, "INVALID"), ("Hk", 4, "INVALID"), ("N", -1, "INVALID"),
    ("C", 0, "INVALID"), ("d", 0, "INVALID"), ("io_dtype", 5, "INVALID"), ("window", -1, "INVALID"),
    ("prefix", -2, "INVALID"), ("scale", 0.0, "INVALID"), ("flags", 8, "INVALID"), ("d", 200, "UNSUPPORTED"),
    ("B", 1 << 23, "UNSUPPORTED"), ("N", 0x7fffffff, "UNSUPPORTED")])
def test_step_descriptor(field, value, status):
    c = Step()
    setattr(c.desc, field, value)
    assert c.call() == getattr(tmm, "ERR_" + status)
    assert tmm.attention_step_workspace_bytes(c.desc) == getattr(tmm, "ERR_" + status)


def test_step_pointers():
    c = Step()
    assert c.ws > 0
    for name in c.names[:-1]:
        assert c.call(**{name: c.p[name] + 8}) == tmm.ERR_INVALID, name
    for name in ("q", "k", "v", "lengths", "out", "k_new", "v_new"):     # (the new ones come together)
        assert c.call(**{name: 0}) == tmm.ERR_INVALID, name
    for out in ("out", "ws", "k", "v"):
        for name in c.names[:-1]:
            if name != out:
                assert c.call(**{out: c.p[name]}) == tmm.ERR_ALIAS, (out, name)
    assert c.call(ws=0) == tmm.ERR_WORKSPACE and c.call(ws_bytes=c.ws - 1) == tmm.ERR_WORKSPACE
    assert tmm.attention_step_workspace_bytes(Step(C=64).desc) == 0
    c.desc.N = 0            # no new tokens: nothing to do, and nothing needed
    assert tmm.attention_step_workspace_bytes(c.desc) == 0 and c.call(ws=0, ws_bytes=0) == tmm.OK


@pytest.mark.parametrize("kind", [Projection, ProjectionBackward])
@pytest.mark.parametrize("field,value,status", [
    ("abi_version", 0, "INVALID"), ("rows", -1, "INVALID"), ("K", 0, "INVALID"), ("O", -3, "INVALID"),
    ("io_dtype", 2, "INVALID"), ("activation", 2, "INVALID"), ("flags", 1, "INVALID"), ("K", (1 << 22) + 1, "UNSUPPORTED"),
    ("rows", 1 << 40, "UNSUPPORTED")])
def test_projection_descriptor(kind, field, value, status):
    c = kind()
    setattr(c.desc, field, value)
    assert c.call() == getattr(tmm, "ERR_" + status)
    if kind is ProjectionBackward:
        assert tmm.projection_backward_workspace_bytes(c.desc) == getattr(tmm, "ERR_" + status)


def test_projection_pointers():
    for c, must, outs in ((Projection(), ("x", "weight", "out"), ("out", "pre")),
                          (ProjectionBackward(), ("x", "weight", "pre", "dout", "dx", "dweight", "dbias"),
                           ("dx", "dweight", "dbias", "ws"))):
        given = [n for n in c.names if n != "ws_bytes"]
        for name in given:
            assert c.call(**{name: c.p[name] + 4}) == tmm.ERR_INVALID, name
        for name in must:
            assert c.call(**{name: 0}) == tmm.ERR_INVALID, name
        for out in outs:
            for name in given:
                if name != out and {out, name} != {"out", "residual"}:
                    assert c.call(**{out: c.p[name]}) == tmm.ERR_ALIAS, (out, name)
    assert Projection().call(out=Projection().p["residual"] + 16) == tmm.ERR_ALIAS     # in place, but not exactly
    c = ProjectionBackward()
    assert c.call(ws=0) == tmm.ERR_WORKSPACE and c.call(ws_bytes=c.ws - 1) == tmm.ERR_WORKSPACE
    c.desc.activation = tmm.ACT_NONE      # no activation, no pre
    assert c.call() == tmm.ERR_INVALID


def test_descriptors_match_the_header():
    """Sizes of the C structures as the compiler lays them out (all fields of 4 bytes, one of 8)."""
    assert ctypes.sizeof(tmm.AttentionDesc) == 44 and ctypes.sizeof(tmm.AttentionStepDesc) == 48
    assert ctypes.sizeof(tmm.ProjectionDesc) == 32


def test_wrappers_refuse_before_the_library():
    import torch
    z = torch.zeros
    q, k = z(2, 4, 5, 8), z(2, 2, 5, 8)
    n = z(2, dtype=torch.int32)
    bad = [lambda: tmm.attention(q, k, k),                                             # right, but on the CPU
           lambda: tmm.attention(q.half(), k.half(), k.half()), lambda: tmm.attention(None, k, k),
           lambda: tmm.attention(q, k, None), lambda: tmm.attention(q, k, z(2, 2, 5, 9)),
           lambda: tmm.attention(q, k.bfloat16(), k), lambda: tmm.attention(q.transpose(1, 2), k, k),
           lambda: tmm.attention(q, k, k, lengths=n.long()), lambda: tmm.attention(q, k, k, lengths=z(3, dtype=torch.int32)),
           lambda: tmm.attention(q, k, k, offsets=n), lambda: tmm.attention(q[0], k[0], k[0]),
           lambda: tmm.attention(q[0], k[0], k[0], offsets=n[:1]), lambda: tmm.attention(q[0], k[0], k[0], offsets=n, lengths=n),
           lambda: tmm.attention(q, k, k, out=z(2, 5, 31)), lambda: tmm.attention(q, k, k, lse_out=z(2, 5, 4)),
           lambda: tmm.attention_backward(q, k, k, z(2, 5, 32), z(2, 4, 5), z(2, 5, 31)),
           lambda: tmm.attention_backward(q, k, k, z(2, 5, 32), None, z(2, 5, 32)),
           lambda: tmm.attention_step(q, k, k, n), lambda: tmm.attention_step(q, k, k, None),
           lambda: tmm.attention_step(q, k, k, n, k_new=k), lambda: tmm.attention_step(q, k, k, n, k_new=k, v_new=q),
           lambda: tmm.attention_step(q[0], k[0], k[0], n), lambda: tmm.projection(z(3, 4), z(5, 4)),
           lambda: tmm.projection(z(3, 4), z(5, 6)), lambda: tmm.projection(z(3, 4), z(5, 4).bfloat16()),
           lambda: tmm.projection(z(3, 4), z(4)), lambda: tmm.projection(z(3, 4), z(5, 4), z(5).bfloat16()),
           lambda: tmm.projection(z(3, 4), z(5, 4), residual=z(3, 4)), lambda: tmm.projection(None, z(5, 4)),
           lambda: tmm.projection_backward(z(3, 4), z(5, 4), z(3, 4)),
           lambda: tmm.projection_backward(z(3, 4), z(5, 4), z(3, 5), activation=tmm.ACT_SILU)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    # key heads that do not divide the query heads: the library's answer, raised by the call
    assert tmm._AttentionPlan((2, 4, 5, 8), (2, 3, 5, 8), torch.float32, None, 0, 0, None).back == tmm.ERR_INVALID
    with pytest.raises(ValueError, match="2\\^31"):
        tmm._AttentionPlan((1, 1, 1 << 32, 8), (1, 1, 1 << 32, 8), torch.float32, None, 0, 0, None)
    with pytest.raises(ValueError, match="2\\^31"):
        tmm._AttentionStepPlan((1, 1, 1, 8), (1, 1, 1 << 32, 8), torch.float32, 0, 0, None)
    with pytest.raises(ValueError, match="2\\^31"):
        tmm._ProjectionPlan((3, 1 << 32), (5, 1 << 32), torch.float32, 0)
