"""Cases of the serving operators and of the stand-alone rotation: what is computed, on what.

Operators (public entry points in ``rope_attention_fwd_b200.binding``):

* ``rope_attn_rotary`` / ``rope_attn_rotary_bwd``: rotary positions of q and k at given
  positions, interleaved or half layout, on part of the head, with frequencies scaled for long
  contexts, and the gradients (the learned log-frequency offsets' among them);
* ``rope_attn_cache_append``: keys (rotated on the way) and values of new tokens into a paged
  cache held in 4 bits, the queries of the same tokens rotated beside them;
* ``rope_attn_cache_read``: rows of that cache as the values they stand for;
* ``rope_attn_cache_attn``: attention of ragged queries over that cache.

The cache.  A page holds ``page`` tokens of every kv head; inside a page, each head has
``page / 16`` blocks of 16 tokens, and a block is [K codes | K pairs | V codes | V pairs]:
codes 4 bits each in the order of the channels (even channel in the low nibble), 16 rows of
d / 2 bytes; pairs (step, lo) in fp16 for every 64 channels, 16 rows of d / 64 pairs.  A value
is lo + step * code.  lo is the group's minimum and step a fifteenth of its range, both rounded
to fp16; the code is the nearest one.
"""
import math
import random

import torch

own = False

GROUP = 64          # channels that share a (step, lo) pair
BLOCK = 16          # tokens of a block
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

_ROPE = dict(rot=0, layout="interleaved", scaling="none", factor=1.0, base=10000.0)
_CACHE = dict(_ROPE, Hq=32, Hkv=8, d=128, page=16, dtype="bf16", causal=True, window=0,
              shape_seed=1)


def listed():
    return [
        # rotation of one token's heads in a decode step: latency
        dict(_ROPE, name="rotary decode 1x8 tokens", op="rotary_fwd", B=1, H=32, Hk=8, n=8, d=128,
             dtype="bf16", pos="far", layout="half", rot=64, scaling="parts", factor=8.0,
             token_major=True),
        # the whole of q and k at the benchmark's own shape
        dict(_ROPE, name="rotary fwd 2x32x8192x128", op="rotary_fwd", B=2, H=32, Hk=32, n=8192,
             d=128, dtype="bf16", pos="order", token_major=False),
        # gradients of a training step at the second workload's shape, learned frequencies
        dict(_ROPE, name="rotary bwd 4x16x2048x64", op="rotary_bwd", B=4, H=16, Hk=16, n=2048,
             d=64, dtype="bf16", pos="order", token_major=False),
        # the same in fp32 on ragged sizes, shared kv heads, part of the head, half layout
        dict(_ROPE, name="rotary bwd f32 odd", op="rotary_bwd", B=3, H=12, Hk=4, n=1021, d=96,
             dtype="f32", pos="far", layout="half", rot=48, scaling="linear", factor=4.0,
             token_major=True),
        # one new token for each of 64 requests
        dict(_CACHE, name="append 64 x 1", op="append", seqs=64, q_min=1, q_max=1, past_min=0,
             past_max=8191),
        # prompts of three requests, ragged
        dict(_CACHE, name="append prompts", op="append", seqs=3, q_min=1500, q_max=4095,
             past_min=0, past_max=700, page=64, layout="half", scaling="parts", factor=4.0),
        # short rows of a small fp32 cache
        dict(_CACHE, name="read small f32", op="read", seqs=5, q_min=1, q_max=77, past_min=0,
             past_max=300, Hq=4, Hkv=2, d=64, page=32, dtype="f32"),
        # whole caches of four requests (moved to another layout or checked)
        dict(_CACHE, name="read 4 caches", op="read", seqs=4, q_min=3000, q_max=8190, past_min=0,
             past_max=0, page=64),
        # one request, one token, a short cache, every head its own keys: latency
        dict(_CACHE, name="attn decode short", op="attn", seqs=1, q_min=1, q_max=1, past_min=512,
             past_max=512, Hq=16, Hkv=16, d=64),
        # decode over ragged caches up to 32768 tokens, shared kv heads
        dict(_CACHE, name="attn decode 16 long", op="attn", seqs=16, q_min=1, q_max=1,
             past_min=100, past_max=32767),
        # fp32, a few tokens of each request at once
        dict(_CACHE, name="attn f32 4 tokens", op="attn", seqs=6, q_min=2, q_max=4, past_min=33,
             past_max=4095, Hq=8, Hkv=2, d=64, page=64, dtype="f32"),
        # a chunk of each of two prompts over their caches
        dict(_CACHE, name="attn prompt chunks", op="attn", seqs=2, q_min=900, q_max=2048,
             past_min=3000, past_max=8192, page=64),
    ]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) )))))


def _draw_rope(rng, d):
    rot = rng.choice([0, 0, d // 2, d - 2 * rng.randint(1, d // 2 - 1)])
    scaling = rng.choice(["none", "linear", "parts"])
    return dict(rot=rot, layout=rng.choice(["interleaved", "half"]), scaling=scaling,
                factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                base=rng.choice([10000.0, 500000.0]))


def draw(rng):
    limit = {"rotary": listed()[1], "cache": listed()[9], "attn": listed()[11]}
    op = rng.choice(["rotary_fwd", "rotary_bwd", "append", "read", "attn", "attn"])
    while True:
        if op.startswith("rotary"):
            d = rng.choice([32, 64, 80, 96, 128])
            H = rng.choice([1, 3, 8, 12, 16, 32])
            c = dict(_draw_rope(rng, d), op=op, B=_spread(rng, 1, 8), H=H,
                     Hk=rng.choice([H, max(1, H // 4), 1]), n=_spread(rng, 1, 8192), d=d,
                     dtype=rng.choice(["bf16", "bf16", "f32"]), pos=rng.choice(["order", "far"]),
                     token_major=rng.random() < 0.5)
            if work(c)["bytes"] <= work(limit["rotary"])["bytes"]:
                return c
            continue
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8, 16])
        c = dict(_draw_rope(rng, d), op=op, seqs=_spread(rng, 1, 64), Hkv=Hkv,
                 Hq=Hkv * rng.choice([1, 2, 3, 4, 7, 8]), d=d,
                 page=rng.choice([16, 32, 64, 128]),
                 dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), causal=True, window=0,
                 shape_seed=rng.randint(1, 10 ** 6))
        if op == "attn":
            c["causal"] = rng.random() < 0.85
            c["window"] = rng.choice([0, 0, 0, _spread(rng, 20, 4096)]) if c["causal"] else 0
            c["q_max"] = rng.choice([1, 1, _spread(rng, 2, 16), _spread(rng, 17, 2048)])
            c["past_max"] = _spread(rng, 1, 32767)
            most = limit["attn"]
        else:
            c["q_max"] = rng.choice([1, _spread(rng, 2, 4096)])
            c["past_max"] = _spread(rng, 1, 8191)
            most = limit["cache"]
        c["q_min"] = max(1, c["q_max"] // 3)
        c["past_min"] = c["past_max"] // 4
        w, top = work(c), work(most)
        kv = sum(p + q for q, p in _lens(c)) * c["Hkv"] * c["d"]
        if (w["flops"] <= top["flops"] or op != "attn") and \
                w["bytes"] <= work(limit["cache"])["bytes"] and kv <= 250000 * 8 * 128:
            return c


# ------------------------------------------------------------------ sizes
def _lens(c):
    """(new tokens, tokens before them) of every request; the first one has the most."""
    r = random.Random(c["shape_seed"])
    return [(c["q_max"], c["past_max"])] + [
        (r.randint(c["q_min"], c["q_max"]), r.randint(c["past_min"], c["past_max"]))
        for _ in range(c["seqs"] - 1)]


def _block_bytes(d):
    return 2 * BLOCK * (d // 2 + 4 * (d // GROUP))


def _pairs(c, q, past):
    """Keys seen, summed over the q rows of a request with `past` tokens before them."""
    L = past + q
    if not c["causal"]:
        return q * L
    if not c["window"]:
        return q * past + q * (q + 1) // 2
    return sum(min(past + i + 1, c["window"]) for i in range(q))


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"].startswith("rotary"):
        x = c["B"] * (c["H"] + c["Hk"]) * c["n"] * c["d"]
        r = c["B"] * (c["H"] + c["Hk"]) * c["n"] * (c["rot"] or c["d"])
        p = 4 * c["B"] * c["n"] if c["pos"] != "order" else 0
        if c["op"] == "rotary_fwd":
            return {"bytes": 2 * e * x + p, "flops": 3 * r}
        # dy read, dx written, and the rotated part of x read for the offsets' gradient
        return {"bytes": 2 * e * x + e * r + p, "flops": 6 * r}
    lens = _lens(c)
    T, d = sum(q for q, _ in lens), c["d"]
    row = d // 2 + 4 * (d // GROUP)
    if c["op"] == "append":    # and the appended rows read back as values
        new = 2 * T * c["Hkv"]
        return {"bytes": 2 * e * T * c["Hq"] * d + 2 * new * (e * d + row),
                "flops": 3 * T * (c["Hq"] + c["Hkv"]) * d + 6 * new * d}
    if c["op"] == "read":
        return {"bytes": 2 * T * c["Hkv"] * (row + e * d), "flops": 4 * T * c["Hkv"] * d}
    seen = 0
    for q, past in lens:
        seen += min(past + q, c["window"] + q - 1) if c["window"] else past + q
    pairs = sum(_pairs(c, q, past) for q, past in lens)
    return {"bytes": 2 * seen * c["Hkv"] * row + T * c["Hq"] * (2 * e * d + 4),
            "flops": 4 * pairs * c["Hq"] * d}


# ------------------------------------------------------------------ frequencies
def _scaled(c):
    """theta_m of the case's base and scaling (no learned offsets), as Python floats."""
    r = c["rot"] or c["d"]
    th = []
    for m in range(r // 2):
        t = c["base"] ** (-2.0 * m / r)
        if c["scaling"] == "linear":
            t = t / c["factor"]
        elif c["scaling"] == "parts":
            # turns of the band over the original context: few -> scaled, many -> kept
            g = (4096.0 * t / (2.0 * math.pi) - 1.0) / (32.0 - 1.0)
            g = min(1.0, max(0.0, g))
            t = (1.0 - g) * t / c["factor"] + g * t
        th.append(t)
    return th


def _amplitude(c):
    return 1.0 + 0.1 * math.log(c["factor"]) if c["scaling"] == "parts" else 1.0


def _spec(c):
    from rope_attention_fwd_b200 import binding as rb
    return rb.rotary_spec(c["d"], base=c["base"], rot_dim=c["rot"] or c["d"], layout=c["layout"],
                          scaling=c["scaling"], factor=c["factor"], orig_len=4096, slow=1.0,
                          fast=32.0, amplitude=_amplitude(c))


# ------------------------------------------------------------------ inputs
def _device():
    return torch.device("cuda")


def _rows(g, n_rows, heads, d, dtype, spread=True):
    """[n_rows, heads, d] activations: normal, some channels of each head larger than others."""
    x = torch.randn((n_rows, heads, d), generator=g, device=_device())
    if spread:
        gain = torch.exp(0.3 * torch.randn((heads, d), generator=g, device=_device()))
        x *= gain
    return x.to(dtype)


def _quantise(x):
    """x [..., d] fp32 -> codes [..., d] (whole numbers in fp32), step and lo [..., d / 64] fp16."""
    y = x.unflatten(-1, (-1, GROUP))
    lo = y.amin(-1).half()
    step = ((y.amax(-1) - lo.float()) * (1.0 / 15.0)).half()
    lo32, step32 = lo.float().unsqueeze(-1), step.float().unsqueeze(-1)
    inv = torch.where(step32 > 0, step32.reciprocal(), torch.zeros_like(step32))
    codes = ((y - lo32) * inv).round().clamp(0, 15)
    return codes.flatten(-2), step, lo


def _pack(codes, step, lo):
    """codes [..., 16, d], step, lo [..., 16, d / 64] -> [..., 16 (d / 2 + 4 d / 64)] bytes."""
    c = codes.to(torch.uint8)
    c = (c[..., 0::2] | (c[..., 1::2] << 4)).flatten(-2)
    p = torch.stack([step, lo], -1).contiguous().view(torch.uint8).flatten(-3)
    return torch.cat([c, p], -1)


def _unpack(part, d):
    """[..., 16 (d / 2 + 4 d / 64)] bytes -> values [..., 16, d] in fp32."""
    n = BLOCK * d // 2
    c = part[..., :n].unflatten(-1, (BLOCK, d // 2))
    codes = torch.stack([c & 15, c >> 4], -1).flatten(-2).float()
    p = part[..., n:].contiguous().view(torch.float16).unflatten(-1, (BLOCK, d // GROUP, 2)).float()
    y = codes.unflatten(-1, (d // GROUP, GROUP))
    return (p[..., 1:] + p[..., :1] * y).flatten(-2)


def prepare(case, seed):
    c = case
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(int(seed))
    r = random.Random(int(seed))
    dt = DTYPES[c["dtype"]]
    s = {"case": c, "theta": torch.tensor(_scaled(c), dtype=torch.float64, device=dev)}
    half = (c["rot"] or c["d"]) // 2
    s["alpha"] = 0.3 * torch.randn((half,), generator=g, device=dev)
    if c["op"].startswith("rotary"):
        B, n, d = c["B"], c["n"], c["d"]
        for name, H in (("q", c["H"]), ("k", c["Hk"]), ("dq", c["H"]), ("dk", c["Hk"])):
            if name[0] == "d" and c["op"] == "rotary_fwd":
                continue
            shape = (B, n, H, d) if c["token_major"] else (B, H, n, d)
            x = torch.randn(shape, generator=g, device=dev).to(dt)
            s[name] = x.transpose(1, 2) if c["token_major"] else x
        s["pos"] = None
        if c["pos"] == "far":
            start = [r.randint(0, 120000) for _ in range(B)]
            s["pos"] = torch.tensor([list(range(a, a + n)) for a in start], dtype=torch.int32,
                                    device=dev)
    else:
        lens = _lens(c)
        T, d, Hkv, page = sum(q for q, _ in lens), c["d"], c["Hkv"], c["page"]
        indptr = [0]
        for q, _ in lens:
            indptr.append(indptr[-1] + q)
        kv = [q + p for q, p in lens]
        need = [-(-x // page) for x in kv]
        ids = list(range(sum(need) + 3))
        r.shuffle(ids)
        table = torch.zeros((len(kv), max(need)), dtype=torch.int32)
        at = 0
        for b, x in enumerate(need):
            table[b, :x] = torch.tensor(ids[at:at + x], dtype=torch.int32)
            at += x
        pages = len(ids)
        s["lens"], s["T"] = lens, T
        s["indptr"] = torch.tensor(indptr, dtype=torch.int32, device=dev)
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=dev)
        s["table"] = table.to(dev)
        s["cache"] = torch.empty((pages, Hkv, page // BLOCK, _block_bytes(d)), dtype=torch.uint8,
                                 device=dev)
        if c["op"] == "append":
            s["cache"].zero_()
            s["k"] = _rows(g, T, Hkv, d, dt)
            s["v"] = _rows(g, T, Hkv, d, dt, False)
            s["q"] = _rows(g, T, c["Hq"], d, dt)
        else:
            gain = torch.exp(0.3 * torch.randn((Hkv, 1, 1, d), generator=g, device=dev))
            some = max(1, (1 << 26) // (Hkv * page * d))
            for a in range(0, pages, some):
                e = min(pages, a + some)
                shape = (e - a, Hkv, page // BLOCK, BLOCK, d)
                k = torch.randn(shape, generator=g, device=dev) * gain
                kp = _pack(*_quantise(k))
                del k
                v = torch.randn(shape, generator=g, device=dev)
                s["cache"][a:e] = torch.cat([kp, _pack(*_quantise(v))], -1)
                del v, kp
            if c["op"] == "attn":
                s["q"] = _rows(g, T, c["Hq"], d, dt)
    if own:
        from rope_attention_fwd_b200 import binding as rb
        s["spec"] = _spec(c)
        if c["op"] in ("rotary_fwd", "append"):
            s["freqs"] = rb.rope_attn_rotary_freqs(s["spec"], s["alpha"])
        if "cache" in s:
            s["plan"] = rb.cache_plan(c["seqs"], s["T"], c["Hq"], c["Hkv"], c["d"], dt,
                                      s["cache"].shape[0], c["page"], s["table"].shape[1],
                                      causal=c["causal"], window=c["window"], max_q=c["q_max"])
            s["ws"] = rb.cache_workspace(s["plan"], dev)
    if c["op"] != "rotary_bwd":   # learned offsets that no longer change
        s["theta"] = s["theta"] * torch.exp(s["alpha"].double())
    return s


# ------------------------------------------------------------------ plain forms
def _angles(theta, pos, amplitude):
    """cos and sin of pos * theta, times the amplitude: [..., half] fp32 from 64-bit angles."""
    phi = pos.double().unsqueeze(-1) * theta
    return (amplitude * torch.cos(phi)).float(), (amplitude * torch.sin(phi)).float()


def _halves(x, c):
    r = c["rot"] or c["d"]
    return (x[..., 0:r:2], x[..., 1:r:2]) if c["layout"] == "interleaved" else \
        (x[..., :r // 2], x[..., r // 2:r])


def _put(y, a, b, c):
    r = c["rot"] or c["d"]
    if c["layout"] == "interleaved":
        y[..., 0:r:2], y[..., 1:r:2] = a, b
    else:
        y[..., :r // 2], y[..., r // 2:r] = a, b
    return y


def _rotate(x, cos, sin, c):
    """x [..., d] fp32, cos and sin [..., half] of its rows; what is not rotated stays."""
    a, b = _halves(x, c)
    return _put(x.clone(), cos * a - sin * b, sin * a + cos * b, c)


def _plain_rotary_fwd(s):
    c = s["case"]
    pos = s["pos"] if s["pos"] is not None else torch.arange(c["n"], device=_device())[None]
    cos, sin = (t.unsqueeze(1) for t in _angles(s["theta"], pos, _amplitude(c)))
    return [_rotate(s[x].float(), cos, sin, c).to(s[x].dtype) for x in ("q", "k")]


def _plain_rotary_bwd(s):
    c = s["case"]
    theta = s["theta"] * torch.exp(s["alpha"].double())
    pos = s["pos"] if s["pos"] is not None else torch.arange(c["n"], device=_device())[None]
    cos, sin = (t.unsqueeze(1) for t in _angles(theta, pos, _amplitude(c)))
    out, torque = [], 0.0
    for x, dy in (("q", "dq"), ("k", "dk")):
        dx = _rotate(s[dy].float(), cos, -sin, c)
        a, b = _halves(s[x].float(), c)
        da, db = _halves(dx, c)
        w = (db * a - da * b).double() * pos.double()[:, None, :, None]
        torque = torque + w.sum((0, 1, 2))
        out.append(dx.to(s[dy].dtype))
    return out + [(theta * torque).float()]


def _places(s):
    """(page, block in the page, row in the block) of every token of the call, and its position."""
    c = s["case"]
    pos, seq = [], []
    for b, (q, past) in enumerate(s["lens"]):
        pos.append(torch.arange(past, past + q, device=_device()))
        seq.append(torch.full((q,), b, device=_device()))
    pos, seq = torch.cat(pos), torch.cat(seq)
    page = s["table"].long()[seq, pos // c["page"]]
    inside = pos % c["page"]
    return page, inside // BLOCK, inside % BLOCK, pos


def _plain_read(s):
    """k, v [T, Hkv, d] of the call's tokens."""
    c = s["case"]
    d, n = c["d"], _block_bytes(c["d"]) // 2
    page, blk, row, _ = _places(s)
    out = []
    for part in (slice(0, n), slice(n, 2 * n)):
        x = s["cache"][page, :, blk][..., part]                       # [T, Hkv, n]
        i = row[:, None, None]
        codes = x[..., :BLOCK * d // 2].unflatten(-1, (BLOCK, d // 2))
        codes = torch.gather(codes, 2, i[..., None].expand(-1, c["Hkv"], 1, d // 2))[:, :, 0]
        pair = x[..., BLOCK * d // 2:].contiguous().view(torch.float16)
        pair = pair.unflatten(-1, (BLOCK, d // GROUP * 2))
        pair = torch.gather(pair, 2, i[..., None].expand(-1, c["Hkv"], 1, d // GROUP * 2))[:, :, 0]
        pair = pair.float().unflatten(-1, (d // GROUP, 2))
        y = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
        y = y.unflatten(-1, (d // GROUP, GROUP))
        out.append((pair[..., 1:] + pair[..., :1] * y).flatten(-2).to(DTYPES[c["dtype"]]))
    return out


def _plain_append(s):
    c = s["case"]
    d = c["d"]
    page, blk, row, pos = _places(s)
    cos, sin = (t.unsqueeze(1) for t in _angles(s["theta"], pos, _amplitude(c)))
    q = _rotate(s["q"].float(), cos, sin, c).to(s["q"].dtype)
    n = _block_bytes(d) // 2
    for at, x in ((0, _rotate(s["k"].float(), cos, sin, c)), (n, s["v"].float())):
        codes, step, lo = _quantise(x)
        codes = codes.to(torch.uint8)
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
        pair = torch.stack([step, lo], -1).flatten(-2).contiguous().view(torch.uint8)
        for first, y in ((at, codes), (at + BLOCK * d // 2, pair)):
            w = y.shape[-1]
            cols = first + row[:, None] * w + torch.arange(w, device=_device())   # [T, w]
            heads = torch.arange(c["Hkv"], device=_device())
            s["cache"][page[:, None, None], heads[None, :, None], blk[:, None, None],
                       cols[:, None, :]] = y
    return [q] + _plain_read(s)


def _visible(c, q, L, rows, keys, device):
    """[len(rows), len(keys)] truth: does row i of the q new ones see key j of L?"""
    i = L - q + rows[:, None]
    j = keys[None, :]
    ok = torch.ones((len(rows), len(keys)), dtype=torch.bool, device=device)
    if c["causal"]:
        ok &= j <= i
        if c["window"]:
            ok &= j > i - c["window"]
    return ok


def _plain_attn(s):
    c = s["case"]
    d, Hkv, G, dev = c["d"], c["Hkv"], c["Hq"] // c["Hkv"], _device()
    o = torch.empty((s["T"], c["Hq"], d), dtype=DTYPES[c["dtype"]], device=dev)
    lse = torch.empty((s["T"], c["Hq"]), dtype=torch.float32, device=dev)
    n, at = _block_bytes(d) // 2, 0
    for b, (q, past) in enumerate(s["lens"]):
        L = past + q
        raw = s["cache"][s["table"][b, :-(-L // c["page"])].long()]
        k, v = (_unpack(raw[..., p], d).transpose(0, 1).reshape(Hkv, -1, d)[:, :L]
                for p in (slice(0, n), slice(n, 2 * n)))
        x = s["q"][at:at + q].float().unflatten(1, (Hkv, G)).permute(1, 2, 0, 3)  # [Hkv, G, q, d]
        seen = _visible(c, q, L, torch.arange(q, device=dev), torch.arange(L, device=dev), dev)
        some = max(1, (1 << 28) // (G * q * L))     # kv heads at once
        for h in range(0, Hkv, some):
            e = min(Hkv, h + some)
            S = torch.matmul(x[h:e], k[h:e, None].transpose(-1, -2)) * (1.0 / math.sqrt(d))
            S = torch.where(seen, S, torch.full_like(S, -math.inf))
            m = S.amax(-1, keepdim=True)
            P = torch.exp(S - torch.where(m == -math.inf, torch.zeros_like(m), m))
            l = P.sum(-1, keepdim=True)
            y = torch.matmul(P, v[h:e, None]) / torch.where(l > 0, l, torch.ones_like(l))
            o[at:at + q, h * G:e * G] = y.permute(2, 0, 1, 3).flatten(1, 2).to(o.dtype)
            lse[at:at + q, h * G:e * G] = (m + torch.log(l))[..., 0].permute(2, 0, 1).flatten(1)
        at += q
    return [o, lse]


_PLAIN = {"rotary_fwd": _plain_rotary_fwd, "rotary_bwd": _plain_rotary_bwd,
          "append": _plain_append, "read": _plain_read, "attn": _plain_attn}


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    from rope_attention_fwd_b200 import binding as rb
    op = s["case"]["op"]
    if op == "rotary_fwd":
        return list(rb.rope_attn_rotary(s["spec"], s["freqs"], s["q"], s["k"], pos=s["pos"]))
    if op == "rotary_bwd":
        # a training step: the offsets have just changed, and with them the frequencies
        freqs = rb.rope_attn_rotary_freqs(s["spec"], s["alpha"])
        return list(rb.rope_attn_rotary_bwd(s["spec"], freqs, s["dq"], s["dk"], q=s["q"],
                                            k=s["k"], pos=s["pos"]))
    batch = (s["table"], s["indptr"], s["kv_len"])
    if op == "append":
        q = rb.rope_attn_cache_append(s["plan"], s["cache"], *batch, s["spec"], s["freqs"],
                                      s["k"], s["v"], q=s["q"], ws=s["ws"])
        k, v = rb.rope_attn_cache_read(s["plan"], s["cache"], *batch, ws=s["ws"])
        return [q, k, v]
    if op == "read":
        return list(rb.rope_attn_cache_read(s["plan"], s["cache"], *batch, ws=s["ws"]))
    return list(rb.rope_attn_cache_attn(s["plan"], s["cache"], *batch, s["q"], ws=s["ws"]))


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_turn(x, theta, pos, c, sign=1.0):
    """x [T, H, d] in 64 bits times exp(i sign pos theta), band by band, as complex numbers."""
    r = c["rot"] or c["d"]
    head, tail = x[..., :r], x[..., r:]
    if c["layout"] == "half":
        z = torch.complex(head[..., :r // 2], head[..., r // 2:])
    else:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], r // 2, 2).contiguous())
    phi = sign * pos.double()[:, None, None] * theta
    z = z * torch.polar(torch.full_like(phi, _amplitude(c)), phi)
    if c["layout"] == "half":
        turned = torch.cat([z.real, z.imag], -1)
    else:
        turned = torch.view_as_real(z).flatten(-2)
    return torch.cat([turned, tail], -1)


def _exact_bits(s, b, L):
    """k, v [Hkv, L, d] of request b in 64 bits, byte by byte."""
    c = s["case"]
    d, Hkv = c["d"], c["Hkv"]
    pages = [int(x) for x in s["table"][b, :-(-L // c["page"])]]
    blocks = torch.cat([s["cache"][p] for p in pages], 1)          # [Hkv, blocks, bytes]
    codes, pairs, got, at = BLOCK * d // 2, 4 * BLOCK * (d // GROUP), [], 0
    for _ in range(2):
        raw = blocks[..., at:at + codes].to(torch.int32)
        par = blocks[..., at + codes:at + codes + pairs].contiguous().view(torch.float16).double()
        at += codes + pairs
        y = torch.empty((Hkv, raw.shape[1], codes * 2), dtype=torch.float64, device=raw.device)
        y[..., 0::2], y[..., 1::2] = (raw % 16).double(), torch.div(
            raw, 16, rounding_mode="floor").double()
        step = par[..., 0::2].repeat_interleave(GROUP, -1)
        lo = par[..., 1::2].repeat_interleave(GROUP, -1)
        got.append((y * step + lo).reshape(Hkv, -1, d)[:, :L])
    return got


def _exact_quantised(x):
    """The values that x [T, H, d] (64 bits) stands as in the cache."""
    T, H, d = x.shape
    y = x.reshape(T, H, d // GROUP, GROUP)
    lo = y.min(-1, keepdim=True).values.to(torch.float16).double()
    step = ((y.max(-1, keepdim=True).values - lo) / 15.0).to(torch.float16).double()
    code = torch.where(step > 0, (y - lo) / torch.where(step > 0, step, torch.ones_like(step)),
                       torch.zeros_like(y))
    return (lo + step * torch.clamp(torch.round(code), 0, 15)).reshape(T, H, d)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    dev = _device()
    if c["op"].startswith("rotary"):
        theta = s["theta"]
        pos = torch.arange(c["n"], device=dev).repeat(c["B"]) if s["pos"] is None else \
            s["pos"].flatten()

        def flat(x):       # [B, H, n, d] -> [B n, H, d]
            return x.transpose(1, 2).reshape(-1, x.shape[1], c["d"]).double()

        def back(y):
            return y.reshape(c["B"], c["n"], y.shape[1], c["d"]).transpose(1, 2)

        if c["op"] == "rotary_fwd":
            return [back(_exact_turn(flat(s[x]), theta, pos, c)) for x in ("q", "k")]
        theta = theta * torch.exp(s["alpha"].double())
        out, dtheta = [], torch.zeros_like(theta)
        for x, dy in (("q", "dq"), ("k", "dk")):
            out.append(back(_exact_turn(flat(s[dy]), theta, pos, c, -1.0)))
            # d(rotated x) / d theta = pos times x turned by a further quarter
            quarter = theta * 0 + math.pi / 2
            y = _exact_turn(flat(s[x]), theta, pos, c)
            turned = _exact_turn(y, quarter, torch.ones_like(pos), c) / _amplitude(c)
            prod = flat(s[dy]) * turned * pos.double()[:, None, None]
            a, b = _halves(prod, c)
            dtheta += (a + b).sum((0, 1))
        return out + [theta * dtheta]
    if c["op"] == "append":
        pos = torch.cat([torch.arange(p, p + q, device=dev) for q, p in s["lens"]])
        q = _exact_turn(s["q"].double(), s["theta"], pos, c)
        k = _exact_turn(s["k"].double(), s["theta"], pos, c)
        return [q, _exact_quantised(k), _exact_quantised(s["v"].double())]
    if c["op"] == "read":
        got = [[], []]
        for b, (q, past) in enumerate(s["lens"]):
            for x, y in zip(got, _exact_bits(s, b, past + q)):
                x.append(y[:, past:].transpose(0, 1))
        return [torch.cat(x) for x in got]
    G, d = c["Hq"] // c["Hkv"], c["d"]
    o = torch.zeros((s["T"], c["Hq"], d), dtype=torch.float64, device=dev)
    lse = torch.zeros((s["T"], c["Hq"]), dtype=torch.float64, device=dev)
    at = 0
    for b, (q, past) in enumerate(s["lens"]):
        L = past + q
        k, v = _exact_bits(s, b, L)
        some = max(1, (1 << 27) // L)               # rows at once
        for head in range(c["Hq"]):
            kh, vh = k[head // G], v[head // G]
            for r0 in range(0, q, some):
                rows = torch.arange(r0, min(q, r0 + some), device=dev)
                S = (s["q"][at + rows, head].double() @ kh.T) / math.sqrt(d)
                seen = _visible(c, q, L, rows, torch.arange(L, device=dev), dev)
                S.masked_fill_(~seen, -math.inf)
                total = torch.logsumexp(S, -1)
                w = torch.exp(S - torch.where(total == -math.inf, 0.0, total)[:, None])
                o[at + rows, head] = w @ vh
                lse[at + rows, head] = total
        at += q
    return [o, lse]
