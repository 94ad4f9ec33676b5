"""Host checks of the serving operators, no GPU: how the attention over the cache is cut into
pieces and what of a batch is followed (tests/csrc/cache_host_check.cpp on csrc/serving.h), the
argument checks of the C ABI before anything is launched, and those of the binding."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import serving_ref as ref
from rope_attention_fwd_b200 import binding as rb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(4096)   # aligned, never dereferenced: validation fails first


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host C++ compiler")
def test_pieces_of_work_faults_and_offsets(tmp_path):
    exe = tmp_path / "cache_host_check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__host__=", "-D__device__=",
                    "-I" + os.path.join(ROOT, "rope_attention_fwd_b200", "csrc"),
                    os.path.join(ROOT, "tests", "csrc", "cache_host_check.cpp"),
                    "-o", str(exe)], check=True, capture_output=True, text=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr


def _plan(**kw):
    a = dict(B=2, T=8, Hq=8, Hkv=2, d=128, dtype=rb.RA_BF16, pages=10, page_size=32, max_pages=4)
    a.update(kw)
    return rb.cache_plan(a.pop("B"), a.pop("T"), a.pop("Hq"), a.pop("Hkv"), a.pop("d"),
                         a.pop("dtype"), a.pop("pages"), a.pop("page_size"), a.pop("max_pages"),
                         **a)


def test_cache_sizes():
    for d, per in ((64, 1152), (128, 2304)):
        assert rb.rope_attn_cache_block_bytes(d) == per == ref.block_bytes(d)
        assert rb.rope_attn_cache_bytes(_plan(d=d)) == 10 * 2 * 2 * per
    assert rb.rope_attn_cache_block_bytes(96) == 0
    # offsets past 32 bits are counted, not wrapped
    assert rb.rope_attn_cache_bytes(_plan(pages=1 << 24, page_size=128)) == (1 << 24) * 2 * 8 * 2304


@pytest.mark.parametrize("bad, code", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hq=7), 1), (dict(page_size=24), 1),
    (dict(page_size=0), 1), (dict(pages=0), 1), (dict(max_pages=0), 1), (dict(window=-1), 1),
    (dict(window=5, causal=False), 1), (dict(scale=float("nan")), 1), (dict(dtype=9), 1),
    (dict(max_q=-1), 1), (dict(scale=1e300), 1), (dict(scale=-0.1), 1),
    (dict(d=96), 2), (dict(d=256), 2), (dict(page_size=8192), 2), (dict(B=65537), 2),
    (dict(Hq=8192, Hkv=2), 2), (dict(max_pages=1 << 30), 2), (dict(T=1 << 40), 2),
    (dict(T=1 << 30, Hq=4096, Hkv=2), 2), (dict(pages=1 << 40), 2),
])
def test_bad_plans_are_refused(bad, code):
    p = _plan(**bad)
    assert rb.rope_attn_cache_bytes(p) == 0 and rb.rope_attn_cache_workspace_bytes(p) == 0
    rows = rb.RaRows(4096, 8, 0, 128, 1024)
    assert rb.lib().rope_attn_cache_attn(ctypes.byref(p), FAKE, FAKE, FAKE, FAKE,
                                         ctypes.byref(rows), FAKE, FAKE, FAKE, 1 << 40,
                                         None) == code


def test_bad_cache_calls_are_refused_before_launch():
    lib, p = rb.lib(), _plan()
    need = rb.rope_attn_cache_workspace_bytes(p)
    q, kv = rb.RaRows(4096, 8, 0, 128, 1024), rb.RaRows(4096, 2, 0, 128, 256)
    by = ctypes.byref
    spec = rb.rotary_spec(128)
    other = rb.rotary_spec(64)

    def attn(rows=q, o=FAKE, lse=FAKE, ws=FAKE, n=need, cache=FAKE, table=FAKE):
        return lib.rope_attn_cache_attn(by(p), cache, table, FAKE, FAKE, by(rows), o, lse, ws, n,
                                        None)

    assert attn(ws=None) == 3 and attn(n=need - 1) == 3 and attn(ws=ctypes.c_void_p(4104)) == 3
    assert attn(cache=None) == 1 and attn(table=None) == 1 and attn(o=None) == 1
    assert attn(lse=None) == 1 and attn(o=ctypes.c_void_p(4098)) == 1
    assert attn(rows=rb.RaRows(4096, 7, 0, 128, 1024)) == 1
    assert attn(rows=rb.RaRows(4096, 8, 0, -128, 1024)) == 1
    assert attn(rows=rb.RaRows(None, 8, 0, 128, 1024)) == 1
    assert attn(rows=rb.RaRows(4097, 8, 0, 128, 1024)) == 1

    def append(k=kv, v=kv, qi=q, qo=q, r=spec, f=FAKE):
        return lib.rope_attn_cache_append(by(p), FAKE, FAKE, FAKE, FAKE, by(r), f, by(k), by(v),
                                          by(qi) if qi else None, by(qo) if qo else None, FAKE,
                                          need, None)

    assert append(r=other) == 1 and append(f=None) == 1 and append(qo=None) == 1
    assert append(qi=None) == 1
    assert append(k=rb.RaRows(4096, 3, 0, 128, 256)) == 1
    # written rows that overlap: heads on top of each other, tokens on top of each other
    assert append(qo=rb.RaRows(1 << 20, 8, 0, 64, 1024)) == 1
    assert append(qo=rb.RaRows(1 << 20, 8, 0, 128, 512)) == 1
    assert append(qo=rb.RaRows(1 << 20, 8, 0, 0, 1024)) == 1
    # in place with other strides
    assert append(qo=rb.RaRows(4096, 8, 0, 1024, 128)) == 1

    def read(k=kv, v=kv):
        return lib.rope_attn_cache_read(by(p), FAKE, FAKE, FAKE, FAKE, by(k), by(v), FAKE, need,
                                        None)

    assert read(k=rb.RaRows(1 << 20, 2, 0, 64, 256)) == 1
    assert read(v=rb.RaRows(1 << 20, 2, 0, 128, 128)) == 1


@pytest.mark.parametrize("bad, code", [
    (dict(d=3), 1), (dict(d=0), 1), (dict(d=64, rot_dim=66), 1), (dict(d=64, rot_dim=3), 1),
    (dict(d=64, rot_dim=0), 1), (dict(d=64, base=0.0), 1), (dict(d=64, base=float("inf")), 1),
    (dict(d=64, scaling="linear", factor=0.0), 1),
    (dict(d=64, scaling="parts", factor=2.0, orig_len=0.0), 1),
    (dict(d=64, scaling="parts", factor=2.0, orig_len=10.0, slow=4.0, fast=4.0), 1),
    (dict(d=64, amplitude=float("nan")), 1), (dict(d=64, fixed_bands=33), 1),
    (dict(d=64, fixed_bands=-1), 1), (dict(d=258), 2),
])
def test_bad_rotary_specs_are_refused(bad, code):
    s = rb.rotary_spec(**bad)
    assert rb.lib().rope_attn_rotary_freqs(ctypes.byref(s), FAKE, FAKE, None) == code
    assert rb.rope_attn_rotary_workspace_bytes(s) == 0


def test_bad_rotary_calls_are_refused_before_launch():
    lib, s, by = rb.lib(), rb.rotary_spec(64), ctypes.byref
    need = rb.rope_attn_rotary_workspace_bytes(s)
    x = rb.RaRows(4096, 4, 4 * 10 * 64, 10 * 64, 64)

    def fwd(i=x, o=x, B=2, n=10, dt=rb.RA_BF16, f=FAKE, k=None, ko=None):
        return lib.rope_attn_rotary(by(s), B, n, dt, f, None, by(i), by(o), k, ko, None)

    assert fwd(B=0) == 1 and fwd(n=0) == 1 and fwd(dt=5) == 1 and fwd(f=None) == 1
    assert fwd(B=1 << 31) == 2 and fwd(B=1 << 20, n=1 << 20) == 2
    assert fwd(k=by(x)) == 1
    assert fwd(o=rb.RaRows(1 << 20, 4, 0, 640, 64)) == 1            # batches overlap
    assert fwd(o=rb.RaRows(1 << 20, 4, 2560, 640, 32)) == 1         # tokens overlap
    assert fwd(o=rb.RaRows(1 << 20, 3, 2560, 640, 64)) == 1         # heads differ
    assert fwd(o=rb.RaRows(4096, 4, 2560, 64, 256)) == 1            # in place, other strides
    assert fwd(i=rb.RaRows(4097, 4, 2560, 640, 64)) == 1
    s.reserved = 1
    assert fwd() == 1
    s.reserved = 0
    o = rb.RaRows(1 << 20, 4, 2560, 640, 64)

    def bwd(dalpha=FAKE, q=x, ws=FAKE, size=need, out=o):
        return lib.rope_attn_rotary_bwd(by(s), 2, 10, rb.RA_BF16, FAKE, None, by(x), by(out), None,
                                        None, by(q) if q else None, None, dalpha, ws, size, None)

    assert bwd(q=None) == 1 and bwd(ws=None) == 3 and bwd(size=need - 1) == 3
    assert bwd(ws=ctypes.c_void_p(4104)) == 3
    assert bwd(out=x) == 1                                           # dq on top of q


def test_binding_refuses_host_tensors_and_bad_names():
    s = rb.rotary_spec(64)
    x = torch.zeros((1, 2, 3, 64))
    with pytest.raises(ValueError, match="CUDA device"):
        rb.rope_attn_rotary(s, torch.zeros(32, dtype=torch.float64), x)
    with pytest.raises(ValueError, match="CUDA device"):
        rb.rope_attn_cache_read(_plan(), torch.zeros(8, dtype=torch.uint8), None, None, None)
    with pytest.raises(ValueError, match="layout"):
        rb.rotary_spec(64, layout="other")
    with pytest.raises(ValueError, match="scaling"):
        rb.rotary_spec(64, scaling="other")


def test_marshal_extension_declines_what_is_not_plain():
    """The C++ marshalling is built, takes no host tensor and no wrong argument: None, which
    sends the call the general way."""
    assert rb._fast is not None, "run python -m rope_attention_fwd_b200.build"
    import ctypes as c
    s, p = rb.rotary_spec(64), _plan()
    x = torch.zeros((1, 2, 3, 64))
    f = torch.zeros(32, dtype=torch.float64)
    for args in ((c.addressof(s), f, x, None, None), (c.addressof(s), f, None, None, None),
                 (c.addressof(s), 3, "x", 5, 1.0), ()):
        assert rb._fast.rotary(*args) is None
    assert rb._fast.rotary_bwd(c.addressof(s), f, x, None, x, None, None) is None
    assert rb._fast.rotary_freqs(c.addressof(s), f) is None
    z = torch.zeros(8, dtype=torch.uint8)
    assert rb._fast.cache_read(c.addressof(p), z, z, z, z, z) is None
    assert rb._fast.cache_attn(c.addressof(p), z, None, z, z, z, z) is None
    assert rb._fast.cache_append(c.addressof(p), z, z, z, z, c.addressof(s), f, z, z, None,
                                 None) is None


class FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return {"rope_attn_cache_bytes": 10 * 2 * 2 * 2304}.get(
                name, 1024 if name.endswith("_bytes") else 0)
        return call


@pytest.fixture
def fake(monkeypatch):
    f = FakeLib()
    monkeypatch.setattr(rb, "lib", lambda: f)
    monkeypatch.setattr(rb, "_stream", lambda device: ctypes.c_void_p(0))
    monkeypatch.setattr(rb, "_fast", None)       # the general way (the extension takes CUDA only)
    monkeypatch.setattr(rb, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(rb, "_serving_device", lambda fn, t: t.get_device())   # -1: host memory
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    return f


def _batch():
    bf = torch.bfloat16
    return dict(plan=_plan(), cache=torch.zeros((10, 2, 2, 2304), dtype=torch.uint8),
                table=torch.zeros((2, 4), dtype=torch.int32),
                indptr=torch.zeros(3, dtype=torch.int32), kv_len=torch.zeros(2, dtype=torch.int32),
                q=torch.zeros((8, 8, 128), dtype=bf), kv=torch.zeros((8, 2, 128), dtype=bf),
                freqs=torch.zeros(64, dtype=torch.float64), ws=torch.zeros(1024, dtype=torch.uint8))


def test_well_formed_serving_calls_reach_the_library(fake):
    t = _batch()
    head = (t["plan"], t["cache"], t["table"], t["indptr"], t["kv_len"])
    spec = rb.rotary_spec(128)
    # a fused q | k | v row: strided views with contiguous channels
    row = torch.zeros((8, 12 * 128), dtype=torch.bfloat16).view(8, 12, 128)
    rb.rope_attn_cache_append(*head, spec, t["freqs"], row[:, 8:10], row[:, 10:], q=row[:, :8],
                              ws=t["ws"])
    rb.rope_attn_cache_append(*head, spec, t["freqs"], t["kv"], t["kv"], ws=t["ws"])
    rb.rope_attn_cache_read(*head, ws=t["ws"])
    o, lse = rb.rope_attn_cache_attn(*head, row[:, :8], ws=t["ws"])
    assert o.shape == (8, 8, 128) and lse.shape == (8, 8) and lse.dtype == torch.float32
    x = torch.zeros((2, 5, 3, 128), dtype=torch.bfloat16).transpose(1, 2)   # token-major
    q, k = rb.rope_attn_rotary(spec, t["freqs"], x, x[:, :1])
    assert q.shape == x.shape and k.shape == (2, 1, 5, 128)
    rb.rope_attn_rotary_bwd(spec, t["freqs"], x, q=x)
    assert rb.rope_attn_rotary_bwd(spec, t["freqs"], x, frozen_alpha=True)[1:] == (None, None)
    names = [c for c in fake.calls if not c.endswith("_bytes")]
    assert names == ["rope_attn_cache_append"] * 2 + ["rope_attn_cache_read",
                     "rope_attn_cache_attn", "rope_attn_rotary", "rope_attn_rotary_bwd",
                     "rope_attn_rotary_bwd"]


def test_malformed_serving_tensors_are_refused_before_any_call(fake):
    t = _batch()
    spec = rb.rotary_spec(128)
    head = (t["plan"], t["cache"], t["table"], t["indptr"], t["kv_len"])
    x = torch.zeros((2, 3, 5, 128))
    f = t["freqs"]

    def with_(i, v):
        return head[:i] + (v,) + head[i + 1:]

    cases = [
        lambda: rb.rope_attn_cache_attn(*head, t["q"].float(), ws=t["ws"]),
        lambda: rb.rope_attn_cache_attn(*head, t["q"][:7], ws=t["ws"]),
        lambda: rb.rope_attn_cache_attn(*head, t["q"].transpose(0, 2).contiguous().transpose(0, 2),
                                        ws=t["ws"]),
        lambda: rb.rope_attn_cache_attn(*with_(1, t["cache"][:9]), t["q"], ws=t["ws"]),
        lambda: rb.rope_attn_cache_attn(*with_(1, t["cache"].to(torch.int8)), t["q"], ws=t["ws"]),
        lambda: rb.rope_attn_cache_attn(*with_(2, t["table"].long()), t["q"], ws=t["ws"]),
        lambda: rb.rope_attn_cache_attn(*with_(2, t["table"][:, :3]), t["q"], ws=t["ws"]),
        lambda: rb.rope_attn_cache_attn(*with_(3, t["indptr"][:2]), t["q"], ws=t["ws"]),
        lambda: rb.rope_attn_cache_attn(*with_(4, t["kv_len"][:1]), t["q"], ws=t["ws"]),
        lambda: rb.rope_attn_cache_attn(*head, t["q"], o=t["q"][:, :4], ws=t["ws"]),
        lambda: rb.rope_attn_cache_append(*head, spec, f, t["kv"], t["q"], ws=t["ws"]),
        lambda: rb.rope_attn_cache_append(*head, spec, f.float(), t["kv"], t["kv"], ws=t["ws"]),
        lambda: rb.rope_attn_cache_read(*head, k=t["kv"].float(), ws=t["ws"]),
        lambda: rb.rope_attn_rotary(spec, f, x.half()),
        lambda: rb.rope_attn_rotary(spec, f, x[..., :64]),
        lambda: rb.rope_attn_rotary(spec, f, x, x[:, :, :4]),
        lambda: rb.rope_attn_rotary(spec, f[:32], x),
        lambda: rb.rope_attn_rotary(spec, f, x, pos=torch.zeros((2, 5), dtype=torch.int64)),
        lambda: rb.rope_attn_rotary(spec, f, x, pos=torch.zeros((2, 4), dtype=torch.int32)),
        lambda: rb.rope_attn_rotary(spec, f, x, q_out=x[:, :2]),
        lambda: rb.rope_attn_rotary_bwd(spec, f, x),
        lambda: rb.rope_attn_rotary_bwd(spec, f, x, x, q=x),
        lambda: rb.rope_attn_rotary_bwd(spec, f, x, q=x.bfloat16()),
        lambda: rb.rope_attn_rotary_freqs(spec, torch.zeros(32)),
    ]
    for i, case in enumerate(cases):
        with pytest.raises(ValueError):
            case()
            pytest.fail(f"case {i} was accepted")
    assert [c for c in fake.calls if not c.endswith("_bytes")] == []


def test_reference_rotation_is_relative_and_its_gradient_matches_differences():
    """The oracle's own pins: scores depend on position differences only (amplitude 1), a half
    layout is the interleaved one with the channels permuted, dalpha matches differences."""
    g = np.random.default_rng(5)
    for layout in ("interleaved", "half"):
        r, d = 12, 20
        al = 0.2 * g.standard_normal(r // 2)
        th = ref.frequencies(r, 100.0, al, "parts", 4.0, 300.0, 1.0, 8.0)
        x, y = g.standard_normal((2, 7, d))
        pos = np.arange(7.0)
        a = (ref.rotate(x, pos, th, layout) * ref.rotate(y, pos + 3, th, layout)).sum(-1)
        b = (ref.rotate(x, pos + 50, th, layout) * ref.rotate(y, pos + 53, th, layout)).sum(-1)
        assert np.allclose(a, b, atol=1e-12)
        f, s = ref.pairs(r, layout)
        perm = np.concatenate([np.stack(ref.pairs(r, layout), -1).reshape(-1), np.arange(r, d)])
        assert np.allclose(ref.rotate(x, pos, th, layout)[:, perm],
                           ref.rotate(x[:, perm], pos, th, "interleaved"))
        dy = g.standard_normal((7, d))
        got, _ = ref.rotary_dalpha(x, dy, pos, th, layout, 1.5)
        for m in range(r // 2):
            e = np.zeros(r // 2)
            e[m] = 1e-6
            hi = (dy * ref.rotate(x, pos, th * np.exp(e), layout, 1.5)).sum()
            lo = (dy * ref.rotate(x, pos, th * np.exp(-e), layout, 1.5)).sum()
            assert abs((hi - lo) / 2e-6 - got[m]) <= 1e-6 * max(1.0, abs(got).max())


def test_reference_quantiser_is_within_half_a_step():
    g = np.random.default_rng(6)
    for d in (64, 128):
        x = (g.standard_normal((50, d)) * np.exp(3 * g.standard_normal((50, 1)))).astype(np.float32)
        x[0], x[1] = 0.0, 7.25
        codes, step, lo = ref.quantise(x)
        y = lo.astype(float).repeat(64, -1) + step.astype(float).repeat(64, -1) * codes
        # half a step, plus what fp16 rounding of lo and step can push past an end of the range
        slack = np.abs(lo).astype(float) * 2.0 ** -11 + 15 * step.astype(float) * 2.0 ** -11 + 1e-6
        assert (np.abs(y - x) <= (0.5 * step.astype(float) + slack).repeat(64, -1)).all()
        assert codes.max() == 15 and codes[0].max() == 0


@pytest.mark.skipif(rb._fast is None, reason="extension not built")
def test_a_plan_and_a_spec_are_not_taken_for_each_other():
    """The extension reads them by address, so the binding looks at what they are."""
    plan, spec, x = _plan(), rb.rotary_spec(128), torch.zeros(1)
    for call in (lambda: rb.rope_attn_cache_attn(spec, x, x, x, x, x, ws=x),
                 lambda: rb.rope_attn_cache_read(spec, x, x, x, x, ws=x),
                 lambda: rb.rope_attn_cache_append(plan, x, x, x, x, plan, x, x, x, ws=x),
                 lambda: rb.rope_attn_rotary(plan, x, x),
                 lambda: rb.rope_attn_rotary_freqs(plan, x),
                 lambda: rb.rope_attn_rotary_bwd(None, x, x)):
        with pytest.raises(TypeError):
            call()
