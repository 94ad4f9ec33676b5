"""The paged 4-bit cache and the attention over it against the float64 oracle (tolerances:
tests/serving_helpers.py; the append's bits against the oracle's quantiser)."""
import numpy as np
import pytest
import torch

from oracle import serving_ref as ref
from rope_attention_fwd_b200 import binding as rb
from serving_helpers import Batch

pytestmark = pytest.mark.gpu

ONE = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 31), (1, 127), (1, 128), (1, 129), (1, 300)]
FEW = [(3, 3), (2, 130), (1, 40), (4, 500), (7, 64), (1, 1)]
MANY = [(65, 65), (40, 333), (1, 129), (130, 131), (17, 400)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq, Hkv, page", [(2, 2, 16), (8, 1, 32), (6, 2, 64), (7, 1, 16),
                                           (32, 2, 48)])
@pytest.mark.parametrize("lens", [ONE, FEW, MANY], ids=["one", "few", "many"])
def test_attention(dtype, d, Hq, Hkv, page, lens):
    b = Batch(lens, Hq, Hkv, d, page, dtype, seed=Hq + d).device()
    o, lse = b.attn()
    assert b.status()[0] == 0
    print("of tolerance", b.check(o, lse))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 5, 16, 100, 127, 128, 1000])
def test_windows(dtype, window):
    b = Batch([(1, 1), (1, 300), (9, 290), (70, 75), (33, 129)], 4, 2, 64, 16, dtype, seed=window,
              window=window).device()
    b.check(*b.attn())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_every_row_sees_every_key_without_causal(dtype, d):
    b = Batch([(1, 0), (3, 1), (5, 200), (90, 33), (2, 0)], 4, 2, d, 32, dtype, seed=d,
              causal=False).device()
    b.check(*b.attn())   # empty caches: o = 0, lse = -inf


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_before_the_cache_see_nothing(dtype):
    """Fewer cached tokens than new ones: the first rows' masks leave nothing."""
    b = Batch([(5, 2), (1, 0), (100, 30), (9, 9)], 4, 1, 64, 16, dtype, seed=4).device()
    b.check(*b.attn())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_caches_are_split_and_joined(dtype):
    b = Batch([(1, 9000), (2, 5001), (1, 3), (1, 20000)], 4, 2, 128, 64, dtype, seed=8).device()
    o, lse = b.attn()
    b.check(o, lse)
    for _ in range(3):   # fixed order: the same bits
        o2, l2 = b.attn()
        assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_scale, v_scale", [(30.0, 1.0), (0.0, 1.0), (1.0, 1000.0), (1.0, 1e-3)])
def test_sharp_flat_large_and_small(dtype, q_scale, v_scale):
    b = Batch([(1, 700), (3, 450), (80, 200)], 4, 2, 128, 16, dtype, seed=11, q_scale=q_scale,
              v_scale=v_scale).device()
    b.check(*b.attn())


def test_more_sequences_than_a_block_has_threads():
    g = np.random.default_rng(2)
    lens = [(int(g.integers(1, 4)), int(g.integers(4, 60))) for _ in range(300)]
    b = Batch(lens, 4, 2, 64, 16, "bf16", seed=2).device()
    b.check(*b.attn())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_last_sequence_stay(dtype):
    b = Batch([(1, 40), (20, 90)], 8, 2, 64, 16, dtype, extra=5).device()
    o = torch.full((b.T, 8, 64), 7.0, dtype=b.dtype, device="cuda")
    lse = torch.full((b.T, 8), 7.0, device="cuda")
    b.attn(o=o, lse=lse)
    b.check(o, lse)
    assert (o[-5:] == 7).all() and (lse[-5:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_query_strides(dtype):
    """Rows of a fused projection, head-major rows and unaligned ones: the same bits."""
    b = Batch([(1, 40), (20, 90), (80, 100)], 8, 2, 64, 16, dtype).device()
    o, lse = b.attn()
    q = b.c["q"]
    for pad in (1, 8):
        wide = torch.zeros((b.T, 8 * 64 + 2 * pad), dtype=b.dtype, device="cuda")
        view = wide[:, pad:pad + 512].unflatten(-1, (8, 64))
        view.copy_(q)
        o2, l2 = rb.rope_attn_cache_attn(*b.head, view, ws=b.c["ws"])
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    hm = q.transpose(0, 1).contiguous().transpose(0, 1)
    o2, l2 = rb.rope_attn_cache_attn(*b.head, hm, ws=b.c["ws"])
    assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_both_ways_of_marshalling_agree(monkeypatch):
    """The extension's and the general way's calls give the same bits, and the same refusals."""
    b = Batch([(1, 40), (20, 90), (80, 100)], 8, 2, 64, 16, "bf16", seed=40).device()
    spec = rb.rotary_spec(64, layout="half")
    alpha = 0.1 * torch.randn(32, device="cuda")
    kv = torch.randn((b.T, 2, 64), device="cuda").bfloat16()
    x = torch.randn((2, 3, 50, 64), device="cuda").bfloat16()
    pos = torch.arange(100, dtype=torch.int32, device="cuda").view(2, 50)
    results = []
    for fast in (rb._fast, None):
        assert fast is not None or results
        monkeypatch.setattr(rb, "_fast", fast)
        f = rb.rope_attn_rotary_freqs(spec, alpha)
        b.c["cache"].copy_(torch.from_numpy(b.cache))
        r = [f, *rb.rope_attn_rotary(spec, f, x, x[:, :1], pos=pos),
             *rb.rope_attn_rotary_bwd(spec, f, x, x[:, :2], q=x, k=x[:, 1:], pos=pos),
             *rb.rope_attn_rotary(spec, f, x)[:1],
             rb.rope_attn_cache_append(*b.head, spec, f, kv, kv, q=b.c["q"], ws=b.c["ws"])]
        r += [b.c["cache"].clone(), *rb.rope_attn_cache_read(*b.head, ws=b.c["ws"]), *b.attn()]
        assert rb.rope_attn_cache_append(*b.head, spec, f, kv, kv, ws=b.c["ws"]) is None
        results.append(r)
        with pytest.raises(ValueError):
            rb.rope_attn_cache_attn(*b.head, b.c["q"].float(), ws=b.c["ws"])
        with pytest.raises(ValueError):
            rb.rope_attn_rotary(spec, f, x, x[:, :, :10])
        with pytest.raises(ValueError):
            rb.rope_attn_cache_read(b.plan, b.c["cache"][1:], *b.head[2:], ws=b.c["ws"])
        small = b.c["ws"][:4096]
        with pytest.raises(rb.RopeAttnError) as e:
            rb.rope_attn_cache_attn(*b.head, b.c["q"], ws=small)
        assert rb.STATUS[e.value.code] == "RA_ERR_WORKSPACE"
    for got, want in zip(*results):
        assert torch.equal(got, want) and got.dtype == want.dtype and got.stride() == want.stride()


def test_host_tensors_are_refused():
    b = Batch([(1, 40)], 4, 2, 64, 16, "bf16").device()
    for i in range(1, 5):
        head = list(b.head)
        head[i] = head[i].cpu()
        with pytest.raises(ValueError):
            rb.rope_attn_cache_attn(*head, b.c["q"], ws=b.c["ws"])
    with pytest.raises(ValueError):
        rb.rope_attn_cache_attn(*b.head, b.c["q"].cpu(), ws=b.c["ws"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_queries_stay_in_their_rows(dtype):
    b = Batch([(1, 40), (4, 700), (80, 90)], 4, 2, 64, 16, dtype, seed=21).device()
    o, lse = (t.clone() for t in b.attn())
    rows = [(0, 1), (2, 3), (30, 0)]
    for t, h in rows:
        b.c["q"][t, h, 5] = float("nan")
    o2, lse2 = b.attn()
    hit = torch.zeros((b.T, 4), dtype=torch.bool, device="cuda")
    for t, h in rows:
        hit[t, h] = True
    assert o2[hit].isnan().all() and lse2[hit].isnan().all()
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])
    assert rb.STATUS[b.status()[0]] == ("RA_ERR_RANGE" if dtype == "bf16" else "RA_OK")


def test_large_queries_are_clamped_and_reported():
    for n, L in ((1, 30), (80, 90)):
        b = Batch([(n, L)], 4, 2, 64, 16, "bf16", seed=22).device()
        b.attn()
        assert b.status()[0] == 0
        b.c["q"][0, 0, 0] = 7e4
        o, lse = b.attn()
        assert rb.STATUS[b.status()[0]] == "RA_ERR_RANGE"
        assert o.isfinite().all() and lse.isfinite().all()


def test_calls_on_two_streams_with_a_workspace_each():
    bs = [Batch([(1, 900), (2, 300), (90, 100)], 8, 2, 128, 16, "bf16", seed=30 + i).device()
          for i in range(2)]
    want = [[t.clone() for t in b.attn()] for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for i, (b, s) in enumerate(zip(bs, streams)):
            with torch.cuda.stream(s):
                got[i].append(b.attn())
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for o, lse in g:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


def test_a_sequence_does_not_depend_on_its_neighbours_contents():
    b = Batch([(1, 300), (3, 500), (70, 90), (1, 40)], 8, 2, 64, 16, "bf16", seed=33).device()
    o, lse = (t.clone() for t in b.attn())
    b.c["q"][1:4] *= 3        # the second sequence's queries
    o2, lse2 = b.attn()
    keep = [0] + list(range(4, b.T))
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], lse2[keep])


def test_scale_is_taken():
    b = Batch([(1, 100), (70, 90)], 4, 2, 64, 16, "bf16", scale=0.05).device()
    b.check(*b.attn())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_batches_are_reported_and_not_followed(dtype):
    """Indices that leave the cache are recorded; the other sequences are unharmed.  (That they
    are never followed is shown on the host: tests/test_cache_host.py.)"""
    lens = [(1, 50), (2, 100), (70, 80), (1, 20)]
    for what, code in (("page", 3), ("length", 2), ("indptr", 1), ("max_q", 1)):
        b = Batch(lens, 4, 2, 64, 16, dtype, seed=3, max_q=69 if what == "max_q" else 0).device()
        bad = 2 if what == "max_q" else 1
        if what == "page":
            b.c["table"][1, 2] = 1 << 20
        elif what == "length":
            b.c["kv_len"][1] = b.table.shape[1] * 16 + 1
        elif what == "indptr":
            b.c["indptr"][4] = b.T + 1
            bad = 3
        o, lse = b.attn()
        status, info = b.status()
        assert rb.STATUS[status] == "RA_ERR_CACHE" and info[1:] == [code, bad], (what, info)
        if what == "page":   # the tokens of the bad page count as masked
            k, v = b._rows()[1]
            k[:, 32:48] = v[:, 32:48] = np.nan
            b.check(o, lse, label=what)
        else:
            b.check(o, lse, skip=(bad,), label=what)
        assert b.status()[0] == 0      # read once, cleared


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_launch_follows_new_lengths(dtype):
    """One captured call replayed with other lengths, tables and queries; two graphs that share
    a workspace, replayed in turn."""
    lens = [[(1, 500), (1, 3), (1, 70)], [(1, 9), (1, 512), (1, 200)], [(1, 1), (1, 1), (1, 1)]]
    bs = [Batch(x, 8, 2, 128, 16, dtype, seed=i, spare=40 - sum(-(-L // 16) for _, L in x) + 40)
          .device() for i, x in enumerate(lens)]
    width = max(b.table.shape[1] for b in bs)
    pages = bs[0].plan.pages
    assert all(b.plan.pages == pages for b in bs)
    plan = rb.cache_plan(3, 3, 8, 2, 128, bs[0].dtype, pages, 16, width, max_q=1)
    t = dict(cache=torch.zeros_like(bs[0].c["cache"]), q=torch.zeros_like(bs[0].c["q"]),
             table=torch.zeros((3, width), dtype=torch.int32, device="cuda"),
             indptr=bs[0].c["indptr"].clone(), kv_len=torch.ones(3, dtype=torch.int32,
                                                                 device="cuda"))
    ws = rb.cache_workspace(plan, "cuda")
    out = [(torch.zeros_like(t["q"]), torch.zeros((3, 8), device="cuda")) for _ in range(2)]
    graphs = []
    for o, lse in out:
        def call():
            rb.rope_attn_cache_attn(plan, t["cache"], t["table"], t["indptr"], t["kv_len"],
                                    t["q"], o=o, lse=lse, ws=ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for b in bs + bs[::-1]:
        t["cache"].copy_(b.c["cache"])
        t["q"].copy_(b.c["q"])
        t["kv_len"].copy_(b.c["kv_len"])
        t["table"][:, :b.table.shape[1]] = b.c["table"]
        for g, (o, lse) in zip(graphs, out):
            o.fill_(9)
            g.replay()
        for o, lse in out:
            b.check(o, lse)


def test_shared_pages_and_another_stream():
    """Two sequences on the same prefix pages, run on a side stream."""
    b = Batch([(1, 64), (1, 80)], 4, 2, 64, 16, "bf16", seed=6).device()
    b.table[1, :4] = b.table[0, :4]
    b.c["table"].copy_(torch.from_numpy(b.table))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, lse = b.attn()
    torch.cuda.current_stream().wait_stream(s)
    b.check(o, lse)


def test_offsets_past_32_bits():
    """Pages beyond 4 GiB of cache."""
    d, Hkv, page = 128, 8, 128
    pages = 31000            # 147456 bytes each: 4.57e9
    lens = [(1, 200), (70, 150)]
    b = Batch(lens, 16, Hkv, d, page, "bf16", seed=1).device()
    big = torch.zeros((pages, Hkv, page // 16, 2304), dtype=torch.uint8, device="cuda")
    last = pages - b.plan.pages
    big[last:] = b.c["cache"]
    plan = rb.cache_plan(2, b.T, 16, Hkv, d, b.dtype, pages, page, b.table.shape[1])
    table = b.c["table"] + last
    o, lse = rb.rope_attn_cache_attn(plan, big, table, b.c["indptr"], b.c["kv_len"], b.c["q"],
                                     ws=b.c["ws"])
    b.check(o, lse)
    spec = rb.rotary_spec(d, rot_dim=2)
    x = torch.randn((b.T, Hkv, d), device="cuda").bfloat16()
    big.zero_()
    rb.rope_attn_cache_append(plan, big, table, b.c["indptr"], b.c["kv_len"], spec,
                              rb.rope_attn_rotary_freqs(spec), x, x, ws=b.c["ws"])
    assert not big[:last].any() and big[last:].any()
    _, v = rb.rope_attn_cache_read(plan, big, table, b.c["indptr"], b.c["kv_len"], ws=b.c["ws"])
    assert (v.float() - x.float()).abs().max() < 0.5
    assert rb.rope_attn_device_status(b.c["ws"])[0] == 0


# ------------------------------------------------------------------ append and read
def _append_case(dtype, d, layout, rot, lens, page, extra=0, seed=0, Hq=6, Hkv=3):
    b = Batch([(n, L) for n, L in lens], Hq, Hkv, d, page, dtype, seed=seed, extra=extra).device()
    g = np.random.default_rng(seed + 100)
    spec = rb.rotary_spec(d, rot_dim=rot, layout=layout, base=1e4, amplitude=1.1)
    alpha = torch.from_numpy(0.2 * g.standard_normal(rot // 2)).float().cuda()
    freqs = rb.rope_attn_rotary_freqs(spec, alpha)
    x = {}
    for name, H in (("k", Hkv), ("v", Hkv), ("q", Hq)):
        x[name] = torch.from_numpy(g.standard_normal((b.T, H, d)) * 2).to(b.dtype).cuda()
    return b, spec, freqs, x


def _rotate32(x, pos, theta, layout, A):
    """The rotation in fp32 with every operation rounded (cos and sin from fp64)."""
    x = x.astype(np.float32)
    a, b = ref.pairs(2 * len(theta), layout)
    phi = pos[:, None, None].astype(np.float64) * theta
    c, s = (A * np.cos(phi)).astype(np.float32), (A * np.sin(phi)).astype(np.float32)
    y = x.copy()
    y[..., a] = c * x[..., a] - s * x[..., b]
    y[..., b] = s * x[..., a] + c * x[..., b]
    return y


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d, rot", [(64, 64), (128, 128), (128, 64), (128, 34), (64, 2), (128, 20)])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_append_writes_the_defined_bytes(dtype, d, rot, layout):
    """The cache after an append, byte for byte (the fp32 arithmetic of the definition done in
    numpy), nothing else touched, and q rotated beside it."""
    lens = [(5, 5), (1, 33), (40, 100), (0, 7), (1, 16), (1, 17)]
    b, spec, freqs, x = _append_case(dtype, d, layout, rot, lens, 32, extra=3, seed=d + rot)
    q_out = torch.full_like(x["q"], 5.0)
    got = rb.rope_attn_cache_append(*b.head, spec, freqs, x["k"], x["v"], q=x["q"], q_out=q_out,
                                    ws=b.c["ws"])
    assert got is q_out and b.status()[0] == 0
    want, theta = b.cache.copy(), freqs.cpu().numpy()
    pos = np.concatenate([np.arange(L - n, L) for n, L in lens]).astype(np.int64)
    used = int(b.indptr[-1])
    k32 = _rotate32(x["k"][:used].float().cpu().numpy(), pos, theta, layout, 1.1)
    v32 = x["v"][:used].float().cpu().numpy()
    half, t = b.cache.shape[-1] // 2, 0
    for s, (n, L) in enumerate(lens):
        for p in range(L - n, L):
            page, at = b.table[s, p // 32], p % 32
            for h in range(3):
                for off, y in ((0, k32), (half, v32)):
                    ref.pack_block(want[page, h, at // 16, off:off + half], at % 16,
                                   *ref.quantise(y[t, h]), d)
            t += 1
    have = b.c["cache"].cpu().numpy()
    # cos and sin agree to the last bit but where fp64 rounds on the other side of an fp32 tie
    # (about one value in 2^28): none here
    assert (have == want).all(), int((have != want).sum())
    q64 = ref.rotate(x["q"][:used].double().cpu().numpy(), pos[:, None], theta, layout, 1.1)
    size = 4 * 2.0 ** -24 * 1.1 * 2 * float(x["q"].abs().max())
    tol = torch.finfo(b.dtype).eps / 2 * abs(q64) + size
    assert (abs(q_out[:used].double().cpu().numpy() - q64) <= tol).all()
    assert (q_out[used:] == 5).all()
    # in place and in another stride order: the same bits
    q2 = x["q"].clone()
    rb.rope_attn_cache_append(*b.head, spec, freqs, x["k"].transpose(0, 1).contiguous()
                              .transpose(0, 1), x["v"], q=q2, q_out=q2, ws=b.c["ws"])
    assert torch.equal(q2[:used], q_out[:used]) and (b.c["cache"].cpu().numpy() == want).all()
    # read back: exactly the values
    k, v = rb.rope_attn_cache_read(*b.head, ws=b.c["ws"])
    kk, vv = ref.unpack_cache(want, d)
    t = 0
    for s, (n, L) in enumerate(lens):
        for got, vals in ((k, kk), (v, vv)):
            w = ref.sequence_rows(vals, b.table[s], L, 32)[:, L - n:].transpose(1, 0, 2)
            g = got[t:t + n].double().cpu().numpy()
            assert (abs(g - w) <= (torch.finfo(b.dtype).eps / 2 + 2.0 ** -24) * abs(w)).all()
        t += n


def test_append_unaligned_rows():
    b, spec, freqs, x = _append_case("bf16", 64, "half", 64, [(9, 20), (3, 3)], 16)
    rb.rope_attn_cache_append(*b.head, spec, freqs, x["k"], x["v"], ws=b.c["ws"])
    want = b.c["cache"].clone()
    b.c["cache"].zero_()
    b.c["cache"].copy_(torch.from_numpy(b.cache))
    views = []
    for n in ("k", "v"):
        wide = torch.zeros((b.T, 3 * 64 + 1), dtype=torch.bfloat16, device="cuda")
        view = wide[:, 1:].unflatten(-1, (3, 64))
        view.copy_(x[n])
        views.append(view)
    rb.rope_attn_cache_append(*b.head, spec, freqs, *views, ws=b.c["ws"])
    assert torch.equal(b.c["cache"], want)
    k = torch.zeros((b.T, 3 * 64 + 1), dtype=torch.bfloat16, device="cuda")
    rb.rope_attn_cache_read(*b.head, k=k[:, 1:].unflatten(-1, (3, 64)), ws=b.c["ws"])
    k2, _ = rb.rope_attn_cache_read(*b.head, ws=b.c["ws"])
    assert torch.equal(k[:, 1:].unflatten(-1, (3, 64)), k2) and not k[:, 0].any()


def test_values_beyond_the_range_are_clamped_and_reported():
    b, spec, freqs, x = _append_case("f32", 64, "interleaved", 2, [(4, 4)], 16)
    x["v"][0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 7e4])
    rb.rope_attn_cache_append(*b.head, spec, freqs, x["k"], x["v"], ws=b.c["ws"])
    assert rb.STATUS[b.status()[0]] == "RA_ERR_RANGE"
    _, v = rb.rope_attn_cache_read(*b.head, ws=b.c["ws"])
    # steps of 8000 between -60000 and 60000
    assert v.isfinite().all() and v[0, 0, 0] == v[0, 0, 3] and abs(v[0, 0, 3] - 6e4) < 100
    assert abs(v[0, 0, 1] + 6e4) < 32 and abs(v[0, 0, 2]) <= 4100
    assert (v[1:] - x["v"][1:]).abs().max() < 1.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_appends_and_reads_are_reported(dtype):
    for what, code, bad in (("page", 3, 0), ("length", 2, 1), ("indptr", 1, 1), ("short", 2, 1)):
        b, spec, freqs, x = _append_case(dtype, 64, "half", 64, [(3, 40), (2, 20)], 16)
        if what == "page":
            b.c["table"][0, 2] = -1
        elif what == "length":
            b.c["kv_len"][1] = 1 << 30
        elif what == "indptr":
            b.c["indptr"][2] = b.T + 1
        else:
            b.c["kv_len"][1] = 1
        before = b.c["cache"].clone()
        rb.rope_attn_cache_append(*b.head, spec, freqs, x["k"], x["v"], ws=b.c["ws"])
        status, info = b.status()
        assert rb.STATUS[status] == "RA_ERR_CACHE" and info[1:] == [code, bad], (what, info)
        k = torch.full((b.T, 3, 64), 3.0, dtype=b.dtype, device="cuda")
        rb.rope_attn_cache_read(*b.head, k=k, ws=b.c["ws"])
        assert rb.STATUS[b.status()[0]] == "RA_ERR_CACHE"
        assert (k[:3] == 0).all() if what == "page" else (k[3:] == 3).all()
        rows = torch.ones(b.plan.pages, dtype=torch.bool)
        rows[b.table[1 - bad].tolist()] = False     # the good sequence's pages
        assert torch.equal(b.c["cache"][rows.cuda()], before[rows.cuda()])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_serving_run(dtype, layout):
    """The operators together, as a server uses them: prompts appended in chunks, then single
    tokens, with attention after every append.  The oracle rotates in float64, quantises by the
    definition and attends to the values."""
    d, Hq, Hkv, page, steps = 64, 8, 2, 16, [(33, 5), (20, 70), (1, 1), (1, 1), (1, 1)]
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = np.random.default_rng(17)
    spec = rb.rotary_spec(d, layout=layout, scaling="parts", factor=4.0, orig_len=64.0, fast=8.0,
                          amplitude=1.05)
    alpha = torch.from_numpy(0.2 * g.standard_normal(d // 2)).float().cuda()
    freqs = rb.rope_attn_rotary_freqs(spec, alpha)
    theta = freqs.cpu().numpy()
    pages, width = 20, 8
    table = torch.from_numpy(g.permutation(pages)[:2 * width].reshape(2, width).astype(np.int32))
    cache, past, kept = None, [0, 0], [[], []]
    for news in steps:
        T = sum(news)
        plan = rb.cache_plan(2, T, Hq, Hkv, d, dt, pages, page, width)
        if cache is None:
            cache = rb.new_cache(plan, "cuda")
            ws = rb.cache_workspace(rb.cache_plan(2, 64, Hq, Hkv, d, dt, pages, page, width,
                                                  max_q=64), "cuda")
            ws = torch.zeros(max(ws.numel(), 1 << 27), dtype=torch.uint8, device="cuda")
        row = torch.from_numpy(g.standard_normal((T, (Hq + 2 * Hkv), d))).to(dt).cuda()
        q, k, v = row[:, :Hq], row[:, Hq:Hq + Hkv], row[:, Hq + Hkv:]
        past = [p + n for p, n in zip(past, news)]
        indptr = torch.tensor([0, news[0], T], dtype=torch.int32, device="cuda")
        kv_len = torch.tensor(past, dtype=torch.int32, device="cuda")
        head = (plan, cache, table.cuda(), indptr, kv_len)
        q_rot = rb.rope_attn_cache_append(*head, spec, freqs, k, v, q=q, ws=ws)
        o, lse = rb.rope_attn_cache_attn(*head, q_rot, ws=ws)
        assert rb.rope_attn_device_status(ws)[0] == 0
        pos = np.concatenate([np.arange(p - n, p) for p, n in zip(past, news)])
        k32 = _rotate32(k.float().cpu().numpy(), pos, theta, layout, 1.05)
        check = Batch.__new__(Batch)
        check.lens, check.d, check.Hq, check.Hkv = list(zip(news, past)), d, Hq, Hkv
        check.dtype, check.causal, check.window, check.scale = dt, True, 0, 0.0
        check.indptr = np.array([0, news[0], T])
        rows, t = [], 0
        for s, n in enumerate(news):
            for y in (k32[t:t + n], v[t:t + n].float().cpu().numpy()):
                codes, step, lo = ref.quantise(y)
                val = lo.astype(np.float64)[..., None] + step.astype(np.float64)[..., None] * \
                    codes.reshape(codes.shape[:-1] + (-1, 64))
                kept[s].append(val.reshape(y.shape))
            t += n
            rows.append(tuple(np.concatenate(kept[s][i::2]).transpose(1, 0, 2) for i in (0, 1)))
        check.check(o, lse, q=q_rot.double().cpu().numpy(), rows=rows, label=str(news))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_output_may_be_the_queries(dtype):
    """Whole items, split ones and (bf16) prompt chunks, d 64 and 128."""
    for d in (64, 128):
        b = Batch([(1, 9000), (3, 200), (1, 1), (70, 900), (2, 0)], 4, 2, d, 32, dtype,
                  seed=d + 1).device()
        o, lse = b.attn()
        q = b.c["q"].clone()
        got, lse2 = rb.rope_attn_cache_attn(*b.head, q, o=q, ws=b.c["ws"])
        assert got.data_ptr() == q.data_ptr()
        assert torch.equal(q, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("B", [32, 33, 600])
def test_many_sequences_of_both_kernels(B):
    """One batch around a warp's lanes and beyond a block's threads: every third sequence has
    more than 64 rows per kv head, the others few, some nothing."""
    g = np.random.default_rng(B)
    lens = []
    for i in range(B):
        n = (3, 1, 2)[i % 3]
        lens.append((n, int(g.integers(0, 260)) if i % 7 else 0))
    b = Batch(lens, 32, 1, 64, 16, "bf16", seed=B).device()
    o, lse = b.attn()
    assert b.status()[0] == 0
    b.check(o, lse)
