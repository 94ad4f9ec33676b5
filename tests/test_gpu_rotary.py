"""rope_attn_rotary and rope_attn_rotary_bwd against the float64 oracle.

Tolerances.  The angle is formed in fp64; cos and sin are rounded to fp32 (2^-24 relative to the
amplitude A), the two products and the sum each once (2^-24): an element differs from the exact
one by at most 4 * 2^-24 A (|x0| + |x1|) (first order, rounded up), plus half a step of the
stored type (eps / 2) relative to the value.  dalpha sums p <dx, J x> in fp64 from fp32 dx (the
same 4 * 2^-24) with two products and a difference rounded to fp32 (3 * 2^-24): 8 * 2^-24 of the
sum of absolute values, plus its own fp32 rounding."""
import numpy as np
import pytest
import torch

from oracle import serving_ref as ref
from rope_attention_fwd_b200 import binding as rb

pytestmark = pytest.mark.gpu
U = 2.0 ** -24

SPECS = {
    "all interleaved": dict(),
    "all half": dict(layout="half"),
    "part half": dict(layout="half", rot=0.5, scaling="parts", factor=8.0, orig_len=256.0,
                      slow=1.0, fast=16.0, amplitude=1.2),
    "odd part": dict(rot=-6, scaling="linear", factor=4.0, base=5e5),
    "odd part half": dict(layout="half", rot=-10, fixed_bands=3),
    "two channels": dict(layout="half", rot=2),
}


def make_spec(name, d):
    kw = dict(SPECS[name])
    rot = kw.pop("rot", None)
    if rot is not None:
        rot = int(d * rot) // 2 * 2 if 0 < rot < 1 else d + rot if rot < 0 else rot
        kw["rot_dim"] = max(2, rot)
    kw["fixed_bands"] = min(kw.get("fixed_bands", 0), (kw.get("rot_dim") or d) // 2)
    spec = rb.rotary_spec(d, **kw)
    ref_kw = dict(base=kw.get("base", 1e4), scaling=kw.get("scaling", "none"),
                  factor=kw.get("factor", 1.0), orig_len=kw.get("orig_len", 0.0),
                  slow=kw.get("slow", 1.0), fast=kw.get("fast", 32.0),
                  fixed_bands=kw["fixed_bands"])
    return spec, kw.get("layout", "interleaved"), kw.get("amplitude", 1.0), ref_kw


def n64(t):
    return t.detach().cpu().double().numpy()


def close_rows(got, want, x, layout, r, A, dtype, label):
    a, b = ref.pairs(r, layout)
    size = np.zeros_like(x)
    size[..., a] = size[..., b] = abs(x[..., a]) + abs(x[..., b])
    tol = torch.finfo(dtype).eps / 2 * abs(want) + 4 * U * A * size * (1 + 2.0 ** -7)
    err = abs(n64(got) - want)
    assert (err <= tol).all(), (label, float((err - tol).max()))
    rest = np.ones(x.shape[-1], bool)
    rest[a] = rest[b] = False
    assert (n64(got)[..., rest] == x[..., rest]).all(), label   # what is not rotated is copied


@pytest.mark.parametrize("spec_name", list(SPECS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B, H, Hk, n, d", [(1, 1, 1, 1, 64), (2, 5, 2, 37, 128), (1, 8, 1, 300, 96),
                                            (3, 2, 2, 19, 10), (1, 3, 3, 7, 256)])
def test_rotation_and_gradients(spec_name, dtype, B, H, Hk, n, d):
    spec, layout, A, kw = make_spec(spec_name, d)
    r = spec.rot_dim
    g = torch.Generator().manual_seed(B * 1000 + H * 100 + n + d)
    alpha = 0.3 * torch.randn(r // 2, generator=g)
    theta = ref.frequencies(r, alpha=n64(alpha), **kw)
    freqs = rb.rope_attn_rotary_freqs(spec, alpha.cuda())
    assert np.allclose(n64(freqs), theta, rtol=1e-13, atol=0)
    th = n64(freqs)
    pos = torch.randint(-2000, 120000, (B, n), generator=g, dtype=torch.int32)
    pos[0, 0] = 0
    t = {k: torch.randn((B, h, n, d), generator=g).to(dtype) for k, h in
         (("q", H), ("k", Hk), ("dq", H), ("dk", Hk))}
    c = {k: x.cuda() for k, x in t.items()}
    for p in (None, pos):
        pn = np.arange(n)[None, None] if p is None else n64(p)[:, None]
        pc = None if p is None else p.cuda()
        qo, ko = rb.rope_attn_rotary(spec, freqs, c["q"], c["k"], pos=pc)
        for got, x in ((qo, t["q"]), (ko, t["k"])):
            close_rows(got, ref.rotate(n64(x), pn, th, layout, A), n64(x), layout, r, A, dtype,
                       "forward")
        dq, dk, dal = rb.rope_attn_rotary_bwd(spec, freqs, c["dq"], c["dk"], q=c["q"], k=c["k"],
                                              pos=pc)
        want, size = 0.0, 0.0
        for got, x, dy in ((dq, t["q"], t["dq"]), (dk, t["k"], t["dk"])):
            close_rows(got, ref.rotate(n64(dy), pn, th, layout, A, -1.0), n64(dy), layout, r, A,
                       dtype, "backward")
            w, s = ref.rotary_dalpha(n64(x), n64(dy), pn, th, layout, A)
            want, size = want + w, size + s * A
        err = abs(n64(dal) - want)
        tol = 8 * U * size + U * abs(want)
        assert (err <= tol).all(), (spec_name, float((err / tol.clip(1e-300)).max()))
        # frozen frequencies: the same rows
        fq, fk, none = rb.rope_attn_rotary_bwd(spec, freqs, c["dq"], c["dk"], pos=pc,
                                               frozen_alpha=True)
        assert none is None and torch.equal(fq, dq) and torch.equal(fk, dk)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_alignment_and_in_place(layout, dtype):
    """Token-major views, rows of a fused projection, unaligned starts, shared (expanded)
    inputs and rotation in place give the bits of the contiguous call."""
    B, H, n, d = 2, 6, 33, 64
    spec = rb.rotary_spec(d, layout=layout)
    freqs = rb.rope_attn_rotary_freqs(spec)
    x = torch.randn((B, H, n, d), device="cuda").to(dtype)
    want, _ = rb.rope_attn_rotary(spec, freqs, x)
    tok = x.transpose(1, 2).contiguous().transpose(1, 2)
    got, _ = rb.rope_attn_rotary(spec, freqs, tok)
    assert torch.equal(got, want) and got.stride() == tok.stride()
    for pad in (1, 8):           # fused rows, and rows that start off a 16-byte boundary
        wide = torch.zeros((B, n, H * d + 2 * pad), dtype=dtype, device="cuda")
        view = wide[..., pad:pad + H * d].unflatten(-1, (H, d)).transpose(1, 2)
        view.copy_(x)
        got, _ = rb.rope_attn_rotary(spec, freqs, view)
        assert torch.equal(got, want), pad
        rb.rope_attn_rotary(spec, freqs, view, q_out=view)
        assert torch.equal(view, want), pad
        assert not wide[..., :pad].any() and not wide[..., pad + H * d:].any()
    one = x[:, :1]
    got, _ = rb.rope_attn_rotary(spec, freqs, one.expand(B, H, n, d))
    assert torch.equal(got, want[:, :1].expand(B, H, n, d))
    y = x.clone()
    rb.rope_attn_rotary(spec, freqs, y, y[:, :0 + 1].clone(), q_out=y)
    assert torch.equal(y, want)
    with pytest.raises(rb.RopeAttnError):
        rb.rope_attn_rotary(spec, freqs, x, q_out=x[:, :1].expand(B, H, n, d))


def test_pass_through_keeps_nan_and_infinities():
    """Channels outside the rotated part are copied bit for bit, whatever they hold."""
    for layout in ("interleaved", "half"):
        for rot in (2, 16, 22):
            spec = rb.rotary_spec(64, rot_dim=rot, layout=layout, amplitude=3.0)
            freqs = rb.rope_attn_rotary_freqs(spec)
            x = torch.randn((1, 2, 9, 64), device="cuda")
            x[..., rot:] = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0] *
                                        16, device="cuda")[:64 - rot]
            y, _ = rb.rope_attn_rotary(spec, freqs, x)
            assert torch.equal(y[..., rot:].contiguous().view(torch.int32),
                               x[..., rot:].contiguous().view(torch.int32))
            assert y[..., :rot].isfinite().all()


def test_gradients_match_differences():
    """dx and dalpha against central differences of L = <w, y> in float64 inputs rounded to
    fp32: h = 2^-6 on a linear form (exact but for rounding) and 2^-8 on alpha."""
    B, H, n, d = 1, 2, 5, 12
    g = torch.Generator().manual_seed(3)
    spec = rb.rotary_spec(d, rot_dim=8, layout="half", base=50.0, amplitude=1.5)
    alpha = (0.2 * torch.randn(4, generator=g)).cuda()
    x = torch.randn((B, H, n, d), generator=g).cuda()
    w = torch.randn((B, H, n, d), generator=g).cuda()

    def loss(x, a):
        y, _ = rb.rope_attn_rotary(spec, rb.rope_attn_rotary_freqs(spec, a), x)
        return float((y.double() * w.double()).sum())

    dx, _, da = rb.rope_attn_rotary_bwd(spec, rb.rope_attn_rotary_freqs(spec, alpha), w, q=x)
    # L is linear in x; its fp32 rounding is at most 5 * 2^-24 of sum |w| |y|
    noise = 5 * U * 1.5 * float((w.abs() * x.abs().amax()).sum()) * 2
    for idx in [(0, 0, 0, 0), (0, 1, 4, 3), (0, 1, 2, 7), (0, 0, 3, 11)]:
        e = torch.zeros_like(x)
        e[idx] = 2.0 ** -6
        num = (loss(x + e, alpha) - loss(x - e, alpha)) / 2.0 ** -5
        assert abs(num - float(dx[idx])) <= noise * 2 ** 6
    for m in range(4):
        e = torch.zeros_like(alpha)
        e[m] = 2.0 ** -8
        num = (loss(x, alpha + e) - loss(x, alpha - e)) / 2.0 ** -7
        # third derivative in log-frequency is at most about (p theta)^3 + 3 (p theta)^2 + p theta
        phi = 4 * 1.5
        trunc = (phi ** 3 + 3 * phi ** 2 + phi) * 1.5 * float((w.abs() * x.abs().amax()).sum()) \
            * 2.0 ** -16 / 6
        assert abs(num - float(da[m])) <= noise * 2 ** 8 + trunc


def test_graph_stream_and_repeat():
    """A captured forward and backward, replayed on new contents and on another stream, give
    the eager bits; two runs give the same bits."""
    spec = rb.rotary_spec(128, layout="half")
    x = torch.randn((2, 4, 65, 128), device="cuda").bfloat16()
    dy = torch.randn_like(x)
    alpha = torch.zeros(64, device="cuda")
    ws = torch.empty(rb.rope_attn_rotary_workspace_bytes(spec), dtype=torch.uint8, device="cuda")

    def step():
        f = rb.rope_attn_rotary_freqs(spec, alpha)
        y, _ = rb.rope_attn_rotary(spec, f, x)
        return (y,) + rb.rope_attn_rotary_bwd(spec, f, dy, q=x, ws=ws)[::2]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    side = torch.cuda.Stream()
    for seed in range(3):
        torch.manual_seed(seed)
        x.copy_(torch.randn_like(x))
        alpha.normal_(0, 0.2)
        want = [t.clone() for t in step()]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.current_stream().wait_stream(side)
        again = step()
        for a, b, c in zip(out, want, again):
            assert torch.equal(a, b) and torch.equal(b, c)


def test_matches_the_attention_forward():
    """Rotating by hand and attending without rotation (every band fixed) is the fused forward:
    the same softmax of the same fp32-rounded operands, fp32 path."""
    B, H, n, d = 1, 2, 70, 64
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn((B, H, n, d), generator=g).cuda() for _ in range(3))
    alpha = (0.3 * torch.randn(d // 2, generator=g)).cuda()
    spec = rb.rotary_spec(d)
    qr, kr = rb.rope_attn_rotary(spec, rb.rope_attn_rotary_freqs(spec, alpha), q, k)
    o1, l1 = rb.rope_attn_fwd(q, k, v, alpha, 1e4, True)
    o2, l2 = rb.rope_attn_fwd(qr, kr, v, alpha, 1e4, True, fixed_bands=d // 2)
    assert (o1 - o2).abs().max() <= 1e-5 and (l1 - l2).abs().max() <= 1e-5
