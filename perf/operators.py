"""The operators around the indexer and the sparse attention, as a model's step uses them: rotary
positions, the rotated and quantised cache append, the read-back of a quantised cache, and dense
attention over prompts.

``run`` makes one pass of an operator: in plain torch where ``own`` is false, through the library's
entry points where it is true. ``exact`` computes the same outputs in 64 bits from the definitions.

Shapes: 128 heads over 576-wide latent rows (512 + 64 rotated) with 64 indexer heads of 128 (64 of
them rotated) are the decode configuration's; 8 heads of 128 in fp32 are the tiny decode's. Prompt
attention runs on up-projected heads (128 + 64 rotated columns for q and k, 128 for v) or on
grouped heads of one width, 8 key heads, whole or cut over several GPUs (16 of the 128 heads).
"""
import math
import random

import torch

own = False

BLOCK = 64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # decode batch of 32: the rotary columns of q (into the 576-wide query) and of the indexer query
        dict(name="rope decode 32", op="rope", type="bf16", T=32, H=128, H_I=64, rot=64, layout="interleaved",
             layout_I="half", pos=1048576, factor=40.0, transpose=False),
        # one prompt chunk of two sequences of 4096 new tokens
        dict(name="rope prompt 8192", op="rope", type="bf16", T=8192, H=128, H_I=64, rot=64, layout="interleaved",
             layout_I="half", pos=65536, factor=40.0, transpose=False),
        # the gradient's direction in fp32, an odd number of rows and heads, whole heads rotated
        dict(name="rope fp32 transpose 1023", op="rope", type="f32", T=1023, H=8, H_I=3, rot=128, layout="half",
             layout_I="interleaved", pos=262144, factor=1.0, transpose=True),
        # decode step: one new token for each of 32 sequences into FP8 records and MXFP8 keys
        dict(name="append decode 32", op="append", mode="mxfp8", kv="fp8", B=32, new=1, most=2048, d=576, d_I=128,
             rot=64, lens=1),
        # prefill chunk: 2 x 4096 new tokens
        dict(name="append chunk 2x4096", op="append", mode="mxfp8", kv="fp8", B=2, new=4096, most=16384, d=576,
             d_I=128, rot=64, lens=2),
        # a cached 64K-token prefix read back for the next chunk of its prompt
        dict(name="read prefix 64K", op="read", mode="mxfp8", kv="fp8", B=1, most=65536, least=65536, d=576, d_I=128,
             lens=3),
        # 33 ragged sequences of a serving batch, bf16 latent rows and block-scaled FP8 keys
        dict(name="read ragged 33", op="read", mode="bf16_kfp8", kv="act", B=33, most=2500, least=0, d=576, d_I=128,
             lens=4),
        # short prompts in fp32, 8 heads on 2 key heads
        dict(name="attn fp32 short", op="attn", type="f32", B=5, most=600, least=1, extra=0, H=8, H_kv=2, d_qk=128,
             d_v=128, lens=5),
        # prompts below the selection's K, packed, one from a single token on; every head up-projected
        dict(name="attn packed 128 heads", op="attn", type="bf16", B=9, most=1100, least=1, extra=0, H=128, H_kv=128,
             d_qk=192, d_v=128, lens=6),
        # one whole prompt with grouped heads: the largest case
        dict(name="attn prompt 8192 grouped", op="attn", type="bf16", B=1, most=8192, least=8192, extra=0, H=32,
             H_kv=8, d_qk=128, d_v=128, lens=7),
        # a chunk of 2048 new tokens behind a cached prefix (16 of the 128 heads)
        dict(name="attn chunk 2048 on 32K", op="attn", type="bf16", B=1, most=2048, least=2048, extra=30720, H=16,
             H_kv=16, d_qk=192, d_v=128, lens=8),
        # single tokens over long contexts of different lengths
        dict(name="attn single tokens 16", op="attn", type="bf16", B=16, most=1, least=1, extra=16000, H=64, H_kv=8,
             d_qk=128, d_v=128, lens=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attn", "attn", "attn"])
    seed = rng.randrange(1 << 20)
    if op == "rope":
        rot = rng.choice([16, 32, 64, 64, 96, 128])
        return dict(op=op, type=rng.choice(["bf16", "bf16", "f32"]), T=_log(rng, 1, 8192), H=rng.choice([1, 7, 8, 16, 64, 128]),
                    H_I=rng.choice([1, 3, 8, 32, 64]), rot=rot, layout=rng.choice(["interleaved", "half"]),
                    layout_I=rng.choice(["interleaved", "half"]), pos=_log(rng, 64, 1 << 20),
                    factor=rng.choice([1.0, 4.0, 40.0]), transpose=rng.random() < 0.3)
    if op in ("append", "read"):
        mode = rng.choice(["f32", "bf16", "bf16_kfp8", "mxfp8"])
        kv = rng.choice(["act", "fp8"]) if mode != "f32" else "act"
        d, d_I = rng.choice([(576, 128), (576, 128), (320, 64), (144, 32)])
        if op == "append":
            new = rng.choice([1, _log(rng, 2, 2048)])
            return dict(op=op, mode=mode, kv=kv, B=_log(rng, 1, 64) if new == 1 else rng.randint(1, 3), new=new,
                        most=new + _log(rng, 1, 4096), d=d, d_I=d_I, rot=rng.choice([16, 32, 64]) if d_I >= 64 else 16,
                        lens=seed)
        return dict(op=op, mode=mode, kv=kv, B=_log(rng, 1, 48), most=_log(rng, 1, 1365), least=0, d=d, d_I=d_I, lens=seed)
    type_ = rng.choice(["bf16", "bf16", "bf16", "f32"])
    H, H_kv = rng.choice([(128, 128), (16, 16), (8, 2), (32, 8), (64, 8), (12, 4), (7, 1), (24, 8)])
    d_qk, d_v = rng.choice([(192, 128), (128, 128), (128, 128), (64, 64), (96, 96), (80, 72)])
    kind = rng.choice(["prompt", "packed", "chunk", "single"])
    least, extra = 1, 0
    if kind == "prompt":
        B, most = 1, _log(rng, 2, 4096 if type_ == "bf16" else 700)
        least = most
    elif kind == "packed":
        B, most = rng.randint(2, 24), _log(rng, 2, 1500 if type_ == "bf16" else 300)
        least = rng.choice([0, 1])
    elif kind == "chunk":
        B, most = rng.randint(1, 4), _log(rng, 2, 1024 if type_ == "bf16" else 64)
        extra = _log(rng, 1, 8192 if type_ == "bf16" else 1024)
    else:
        B, most, extra = _log(rng, 1, 64), 1, _log(rng, 1, 16384 if type_ == "bf16" else 2048)
    while B * H * most * (most + extra) > (1 << 30) or B * H_kv * (most + extra) > (1 << 21):
        most, extra, least = max(1, most // 2), extra // 2, min(least, 1) if kind != "prompt" else max(1, most // 2)
    return dict(op="attn", type=type_, B=B, most=most, least=least, extra=extra, H=H, H_kv=H_kv, d_qk=d_qk, d_v=d_v,
                lens=seed)


def lengths(case):
    """The batch's lengths, a part of the case: spread between `least` and `most`, the longest first come."""
    r = random.Random(case["lens"])
    most, least = case["most"], case.get("least", case.get("new", 1))
    n = [most] + [r.randint(least, most) for _ in range(case["B"] - 1)]
    r.shuffle(n)
    return n


def contexts(case, n):
    """Keys that stand before each sequence's queries (a cached prefix): up to `extra`."""
    r = random.Random(case["lens"] + 1)
    e = case["extra"]
    x = [e if case["B"] == 1 else r.randint(0, e) for _ in n]
    if e and case["B"] > 1:
        x[r.randrange(len(x))] = e
    return [a + b for a, b in zip(n, x)]


def starts(n):
    s = [0]
    for v in n:
        s.append(s[-1] + v)
    return s


# ----------------------------------------------------------------------------------------- inputs

def frequencies(rot, base, factor, original):
    """rot / 2 angular frequencies (radians per position, float64), stretched for contexts `factor` times
    the trained length: slow pairs are divided by the factor, fast ones stay, a ramp between them."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot)
    if factor == 1.0:
        return f
    turn = lambda b: rot * math.log(original / (b * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    low, high = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), rot - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp)


def _tables(n, g, spare=3):
    """A shuffled block table for sequences of n positions: (table on the GPU, number of blocks)."""
    blocks = [(v + BLOCK - 1) // BLOCK for v in n]
    total, width = sum(blocks) + spare, max(1, max(blocks))
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = torch.full((len(n), width), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(width, device="cuda")
    nb = torch.tensor(blocks, device="cuda")
    first = torch.tensor(starts(blocks)[:-1], device="cuda")
    used = col[None] < nb[:, None]
    src = (first[:, None] + col[None]).clamp(max=total - 1)
    return torch.where(used, perm[src], at), total


def _codes(shape, g):
    """Finite e4m3 codes of either sign, as bytes."""
    c = torch.randint(0, 127, shape, generator=g, device="cuda", dtype=torch.int16)
    s = torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.int16)
    return (c + 128 * s).to(torch.uint8)


def record_bytes(d):
    return (d + 4 * ((d + 127) // 128) + 15) // 16 * 16


def _caches(case, blocks, g):
    d, d_I, mode = case["d"], case["d_I"], case["mode"]
    act = torch.float32 if mode == "f32" else torch.bfloat16
    if case["kv"] == "fp8":
        tiles = (d + 127) // 128
        kv = torch.zeros((blocks, BLOCK, record_bytes(d)), dtype=torch.uint8, device="cuda")
        kv[..., :d] = _codes((blocks, BLOCK, d), g)
        sc = torch.rand((blocks, BLOCK, tiles), generator=g, device="cuda") * 0.01 + 0.005
        kv[..., d:d + 4 * tiles] = sc.view(torch.uint8)
    else:
        kv = torch.randn((blocks, BLOCK, d), generator=g, device="cuda").to(act)
    scale = None
    if mode == "bf16_kfp8":
        k = _codes((blocks, BLOCK, d_I), g)
        scale = torch.rand((blocks,), generator=g, device="cuda") * 0.01 + 0.005
    elif mode == "mxfp8":
        k = _codes((blocks, BLOCK, d_I), g)
        scale = torch.randint(117, 121, (blocks, BLOCK, d_I // 32), generator=g, device="cuda").to(torch.uint8)
    else:
        k = torch.randn((blocks, BLOCK, d_I), generator=g, device="cuda").to(act)
    return k, scale, kv


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    op = case["op"]
    s = dict(case=case)
    if op == "rope":
        t, T, rot = DTYPES[case["type"]], case["T"], case["rot"]
        s["freq"] = frequencies(rot, 10000.0, case["factor"], 4096).cuda()
        s["scale"] = 0.1 * math.log(case["factor"]) + 1.0
        s["pos"] = torch.randint(0, case["pos"], (T,), generator=g, device="cuda").to(torch.int32)
        # the projection's heads hold 128 columns without positions, then the rotated ones; the rotated
        # ones go to the tail of the query's wide heads
        s["x"] = randn(T, case["H"], 128 + rot).to(t)
        s["q"] = randn(T, case["H"], 512 + rot).to(t)
        s["x_I"] = randn(T, case["H_I"], 64 + rot).to(t)
        s["q_I"] = randn(T, case["H_I"], 64 + rot).to(t)
        return s
    if op == "attn":
        n = lengths(case)
        m = contexts(case, n)
        t = DTYPES[case["type"]]
        s.update(n=n, m=m, cu_q=ints(starts(n)), cu_k=ints(starts(m)), sm_scale=case["d_qk"] ** -0.5)
        s["q"] = randn(sum(n), case["H"], case["d_qk"]).to(t)
        s["k"] = randn(sum(m), case["H_kv"], case["d_qk"]).to(t)
        s["v"] = randn(sum(m), case["H_kv"], case["d_v"]).to(t)
        s["scratch"] = torch.zeros(128 << 20, dtype=torch.uint8, device="cuda")
        return s
    n = lengths(case)
    act = torch.float32 if case["mode"] == "f32" else torch.bfloat16
    s["table"], s["blocks"] = _tables(n, g)
    s["k"], s["k_scale"], s["kv"] = _caches(case, s["blocks"], g)
    s["n"], s["seq_lens"] = n, ints(n)
    s["scratch"] = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    if op == "append":
        new, T = case["new"], case["new"] * case["B"]
        s["freq"] = frequencies(case["rot"], 10000.0, 40.0, 4096).cuda()
        s["q_seq"] = ints([b for b in range(case["B"]) for _ in range(new)])
        s["q_pos"] = ints([v - new + j for v in n for j in range(new)])
        s["k_new"], s["kv_new"] = (3 * randn(T, case["d_I"])).to(act), randn(T, case["d"]).to(act)
    else:
        s["cu"] = ints(starts(n))
        s["rows"] = sum(n)
        s["k_out"] = torch.empty((sum(n), case["d_I"]), dtype=act, device="cuda")
        s["kv_out"] = torch.empty((sum(n), case["d"]), dtype=act, device="cuda")
    return s


# ------------------------------------------------------------------------------------- plain forms

def _rotate(x, pos, freq, layout, scale, transpose):
    """x [T, heads, rot] in fp32, its pairs turned by pos * freq."""
    a = pos.double()[:, None] * freq
    c, s = (scale * a.cos()).float()[:, None], (scale * a.sin()).float()[:, None]
    s = -s if transpose else s
    if layout == "half":
        u, v = x.float().chunk(2, dim=-1)
        return torch.cat((u * c - v * s, u * s + v * c), dim=-1)
    u, v = x.float()[..., 0::2], x.float()[..., 1::2]
    return torch.stack((u * c - v * s, u * s + v * c), dim=-1).flatten(-2)


def _plain_rope(s):
    c = s["case"]
    rot = c["rot"]
    s["q"][..., 512:] = _rotate(s["x"][..., 128:], s["pos"], s["freq"], c["layout"], s["scale"], c["transpose"])
    s["q_I"][..., :rot] = _rotate(s["x_I"][..., :rot], s["pos"], s["freq"], c["layout_I"], s["scale"], c["transpose"])
    return [s["q"][..., 512:], s["q_I"][..., :rot]]


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _tile_scale(x):
    amax = x.abs().amax(dim=-1, keepdim=True)
    return torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))


def _written(s):
    """The caches as outputs: codes and scales as the values they stand for."""
    c = s["case"]
    d = c["d"]
    out = {}
    if c["kv"] == "fp8":
        out["kv"] = s["kv"][..., :d].view(torch.float8_e4m3fn)
        out["kv_scale"] = s["kv"][..., d:d + 4 * ((d + 127) // 128)].view(torch.float32)
    else:
        out["kv"] = s["kv"]
    out["k"] = s["k"].view(torch.float8_e4m3fn) if s["k_scale"] is not None else s["k"]
    if c["mode"] == "bf16_kfp8":
        out["k_scale"] = s["k_scale"]
    elif c["mode"] == "mxfp8":
        out["k_scale"] = s["k_scale"].view(torch.float8_e8m0fnu)
    return out


def _plain_append(s):
    c = s["case"]
    d, d_I, rot = c["d"], c["d_I"], c["rot"]
    k, kv = s["k_new"].float(), s["kv_new"].float()
    kv[:, d - rot:] = _rotate(kv[:, None, d - rot:], s["q_pos"], s["freq"], "interleaved", 1.0, False)[:, 0]
    k[:, :rot] = _rotate(k[:, None, :rot], s["q_pos"], s["freq"], "half", 1.0, False)[:, 0]
    seq, pos = s["q_seq"].long(), s["q_pos"].long()
    blk = s["table"][seq, pos // BLOCK].long()
    row = blk * BLOCK + pos % BLOCK
    if c["kv"] == "fp8":
        tiles = (d + 127) // 128
        x = torch.nn.functional.pad(kv, (0, 128 * tiles - d)).view(-1, tiles, 128)
        sc = _tile_scale(x)
        flat = s["kv"].view(-1, record_bytes(d))
        rec = torch.zeros((len(row), record_bytes(d)), dtype=torch.uint8, device="cuda")
        rec[:, :d] = _e4m3(x / sc).view(-1, 128 * tiles)[:, :d]
        rec[:, d:d + 4 * tiles] = sc.view(-1, tiles).contiguous().view(torch.uint8)
        flat[row] = rec
    else:
        s["kv"].view(-1, d)[row] = kv.to(s["kv"].dtype)
    if c["mode"] == "mxfp8":
        x = k.view(-1, d_I // 32, 32)
        amax = x.abs().amax(dim=-1)
        X = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - 8, -127).clamp(min=-127)
        s["k"].view(-1, d_I)[row] = _e4m3(torch.ldexp(x, -X[..., None])).view(-1, d_I)
        s["k_scale"].view(-1, d_I // 32)[row] = (X + 127).to(torch.uint8)
    elif c["mode"] == "bf16_kfp8":
        # every block that gets new tokens is quantised anew, its earlier tokens from their codes
        touched = torch.zeros(s["blocks"], dtype=torch.bool, device="cuda")
        touched[blk] = True
        fresh = torch.zeros(s["blocks"] * BLOCK, dtype=torch.bool, device="cuda")
        fresh[row] = True
        first = torch.full((s["blocks"],), BLOCK, dtype=torch.int64, device="cuda")
        first.scatter_reduce_(0, blk, pos % BLOCK, "amin")
        old = torch.arange(BLOCK, device="cuda")[None] < first[:, None]
        x = s["k"].view(torch.float8_e4m3fn).float() * s["k_scale"][:, None, None]
        x.view(-1, d_I)[row] = k
        live = (old | fresh.view(-1, BLOCK)) & touched[:, None]
        amax = torch.where(live[..., None], x.abs(), 0.0).amax(dim=(1, 2))
        sc = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        s["k"].copy_(torch.where(live[..., None], _e4m3(x / sc[:, None, None]), s["k"]))
        s["k_scale"].copy_(torch.where(touched, sc, s["k_scale"]))
    else:
        s["k"].view(-1, d_I)[row] = k.to(s["k"].dtype)
    return _written(s)


def _plain_read(s):
    c = s["case"]
    d, d_I = c["d"], c["d_I"]
    r = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), r, right=True)
    pos = r - s["cu"].long()[seq]
    blk = s["table"][seq, pos // BLOCK].long()
    row = blk * BLOCK + pos % BLOCK
    if c["kv"] == "fp8":
        rec = s["kv"].view(-1, record_bytes(d))[row]
        sc = rec[:, d:d + 4 * ((d + 127) // 128)].contiguous().view(torch.float32)
        kv = rec[:, :d].contiguous().view(torch.float8_e4m3fn).float() * sc.repeat_interleave(128, dim=1)[:, :d]
    else:
        kv = s["kv"].view(-1, d)[row]
    k = s["k"].view(-1, d_I)[row]
    if c["mode"] == "bf16_kfp8":
        k = k.view(torch.float8_e4m3fn).float() * s["k_scale"][blk][:, None]
    elif c["mode"] == "mxfp8":
        X = s["k_scale"].view(-1, d_I // 32)[row].float() - 127.0
        k = k.view(torch.float8_e4m3fn).float() * torch.exp2(X).repeat_interleave(32, dim=1)
    s["k_out"].copy_(k)
    s["kv_out"].copy_(kv)
    return [s["k_out"], s["kv_out"]]


def _padded(x, cu, most):
    """Packed rows [R, H, d] as fp32 [B, H, most, d] (rows past a sequence's end repeat another row)."""
    i = cu[:-1].long()[:, None] + torch.arange(most, device="cuda")[None]
    return x[i.clamp(max=max(0, x.shape[0] - 1))].float().transpose(1, 2)


def _plain_attn(s):
    c = s["case"]
    H, G = c["H"], c["H"] // c["H_kv"]
    nq, nk = s["cu_q"].diff(), s["cu_k"].diff()
    Lq, Lk = max(s["n"]), max(s["m"])
    q, k, v = _padded(s["q"], s["cu_q"], Lq), _padded(s["k"], s["cu_k"], Lk), _padded(s["v"], s["cu_k"], Lk)
    B = q.shape[0]
    z = (q * s["sm_scale"]).reshape(B, c["H_kv"], G * Lq, -1) @ k.transpose(-1, -2)
    z = z.view(B, c["H_kv"], G, Lq, Lk)
    i, j = torch.arange(Lq, device="cuda")[:, None], torch.arange(Lk, device="cuda")[None]
    seen = (j <= i + (nk - nq)[:, None, None]) & (j < nk[:, None, None])
    z.masked_fill_(~seen[:, None, None], -math.inf)
    m = z.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = z.sub_(m).exp_()
    l = p.sum(dim=-1, keepdim=True)
    o = (p.view(B, c["H_kv"], G * Lq, Lk) @ v).view(B, c["H_kv"], G, Lq, -1)
    o = o / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + l.log()).squeeze(-1)
    live = torch.arange(Lq, device="cuda")[None] < nq[:, None]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, Lq, H, -1)[live]
    lse = lse.permute(0, 3, 1, 2).reshape(B, Lq, H)[live]
    return [o.to(s["q"].dtype), lse]


# ------------------------------------------------------------------------------- the library's calls

def _own_rope(s):
    import indexer_top_sparse_paged_gb300 as dsa
    c = s["case"]
    rot = c["rot"]
    out = [s["q"][..., 512:], s["q_I"][..., :rot]]
    return dsa.rope([s["x"][..., 128:], s["x_I"][..., :rot]], s["freq"], q_pos=s["pos"], layout=[c["layout"], c["layout_I"]],
                    out=out, scale=s["scale"], transpose=c["transpose"])


def _dims(s):
    import indexer_top_sparse_paged_gb300 as dsa
    c = s["case"]
    return dsa.make_dims(c["mode"], c["B"], s["table"].shape[1], s["blocks"], 64, c["d_I"], 128, c["d"], c["d"] - 64, 2048,
                         kv=c["kv"])


def _own_append(s):
    import indexer_top_sparse_paged_gb300 as dsa
    c = s["case"]
    dsa.cache_append_rope(_dims(s), s["freq"], s["k_new"], s["kv_new"], s["table"], s["seq_lens"], s["k"], s["k_scale"],
                          s["kv"], s["q_seq"], s["q_pos"], k_offset=0, k_layout="half", kv_offset=c["d"] - c["rot"],
                          kv_layout="interleaved", ws=s["scratch"])
    return _written(s)


def _own_read(s):
    import indexer_top_sparse_paged_gb300 as dsa
    return list(dsa.cache_read(_dims(s), s["k"], s["k_scale"], s["kv"], s["table"], s["seq_lens"], s["cu"], s["rows"],
                               k_out=s["k_out"], kv_out=s["kv_out"], ws=s["scratch"]))


def _own_attn(s):
    import indexer_top_sparse_paged_gb300 as dsa
    dims = dsa.prompt_dims(s["q"], s["k"], s["v"], len(s["n"]), causal=True)
    return list(dsa.prompt_attn(dims, s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["sm_scale"], ws=s["scratch"]))


def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "read": _own_read, "attn": _own_attn}[op](s)
    return {"rope": _plain_rope, "append": _plain_append, "read": _plain_read, "attn": _plain_attn}[op](s)


# --------------------------------------------------------------------------------- what a pass needs

def work(case):
    op = case["op"]
    if op == "rope":
        e = 4 if case["type"] == "f32" else 2
        n = case["T"] * (case["H"] + case["H_I"]) * case["rot"]
        return {"bytes": 2 * n * e + 4 * case["T"], "flops": 3 * n}
    if op == "attn":
        n = lengths(case)
        m = contexts(case, n)
        e = 4 if case["type"] == "f32" else 2
        pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(n, m))
        H, H_kv, d, dv = case["H"], case["H_kv"], case["d_qk"], case["d_v"]
        return {"bytes": e * (sum(n) * H * (d + dv) + sum(m) * H_kv * (d + dv)) + 4 * sum(n) * H,
                "flops": 2 * pairs * H * (d + dv)}
    mode, d, d_I = case["mode"], case["d"], case["d_I"]
    act = 4 if mode == "f32" else 2
    row = (record_bytes(d) if case["kv"] == "fp8" else d * act)
    row += d_I * act if mode in ("f32", "bf16") else d_I if mode == "bf16_kfp8" else d_I + d_I // 32
    n = case["B"] * case["new"] if op == "append" else sum(lengths(case))
    return {"bytes": max(1, n) * (row + (d + d_I) * act), "flops": max(1, n) * 4 * (d + d_I)}


# ------------------------------------------------------------------------------------------ 64 bits

def _turned(x, pos, freq, layout, scale, transpose):
    """The pairs as complex numbers times scale * e^(i angle)."""
    x = x.double()
    h = x.shape[-1] // 2
    z = torch.view_as_complex(x.unflatten(-1, (h, 2)).contiguous()) if layout == "interleaved" else torch.complex(x[..., :h], x[..., h:])
    w = torch.polar(torch.full((len(pos), h), float(scale), dtype=torch.float64, device=x.device), torch.outer(pos.double(), freq))
    z = z * (w.conj() if transpose else w)[:, None]
    return torch.view_as_real(z).flatten(-2) if layout == "interleaved" else torch.cat((z.real, z.imag), -1)


def _nearest_e4m3(x):
    """The e4m3 value nearest to x (ties to the even code), saturating, by search in the ordered table."""
    table = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(table, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - table[lo], table[hi] - a
    pick = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return table[pick] * torch.where(x < 0, -1.0, 1.0)


def _exact_attn(s):
    outs, lses = [], []
    c = s["case"]
    G, a, b = c["H"] // c["H_kv"], 0, 0
    for n, m in zip(s["n"], s["m"]):
        o = torch.zeros((n, c["H"], c["d_v"]), dtype=torch.float64, device="cuda")
        e = torch.full((n, c["H"]), -math.inf, dtype=torch.float64, device="cuda")
        if n and m:
            hidden = torch.ones((n, m), dtype=torch.bool, device="cuda").triu(m - n + 1)
            for h in range(c["H"]):
                q, k, v = s["q"][a:a + n, h].double(), s["k"][b:b + m, h // G].double(), s["v"][b:b + m, h // G].double()
                z = ((q @ k.T) * s["sm_scale"]).masked_fill(hidden, -math.inf)
                e[:, h] = torch.logsumexp(z, dim=-1)
                o[:, h] = torch.nan_to_num(torch.softmax(z, dim=-1)) @ v
        outs.append(o)
        lses.append(e)
        a, b = a + n, b + m
    return [torch.cat(outs), torch.cat(lses)]


def _exact_append(s):
    c = s["case"]
    d, d_I, rot = c["d"], c["d_I"], c["rot"]
    k, kv = s["k_new"].double(), s["kv_new"].double()
    kv = torch.cat((kv[:, :d - rot], _turned(kv[:, None, d - rot:], s["q_pos"], s["freq"], "interleaved", 1.0, False)[:, 0]), 1)
    k = torch.cat((_turned(k[:, None, :rot], s["q_pos"], s["freq"], "half", 1.0, False)[:, 0], k[:, rot:]), 1)
    pos = s["q_pos"].long()
    blk = s["table"][s["q_seq"].long(), pos // BLOCK].long()
    slot = pos % BLOCK
    out = {name: v.double() for name, v in _written(s).items()}
    tiles = (d + 127) // 128
    if c["kv"] == "fp8":
        for j in range(tiles):
            x = kv[:, 128 * j:128 * j + 128]
            top = x.abs().amax(1)
            sc = torch.where(top > 0, top / 448.0, 1.0)
            out["kv"][blk, slot, 128 * j:128 * j + 128] = _nearest_e4m3(x / sc[:, None])
            out["kv_scale"][blk, slot, j] = sc
    else:
        out["kv"][blk, slot] = kv
    if c["mode"] == "mxfp8":
        for j in range(d_I // 32):
            x = k[:, 32 * j:32 * j + 32]
            top = x.abs().amax(1)
            X = torch.round(torch.log2(top.clamp(min=2.0 ** -140)))  # then down to the power of two not above it
            X = (torch.where(torch.exp2(X) > top, X - 1, X) - 8).clamp(min=-127)
            out["k"][blk, slot, 32 * j:32 * j + 32] = _nearest_e4m3(x * torch.exp2(-X)[:, None])
            out["k_scale"][blk, slot, j] = torch.exp2(X)
    elif c["mode"] == "bf16_kfp8":
        new = c["new"]
        for b, n in enumerate(s["n"]):
            for lb in range((n - new) // BLOCK, (n - 1) // BLOCK + 1):
                at = int(s["table"][b, lb])
                lo, hi = max(n - new, lb * BLOCK), min(n, (lb + 1) * BLOCK)
                x = torch.cat((out["k"][at, :lo - lb * BLOCK] * out["k_scale"][at], k[b * new + lo - (n - new):b * new + hi - (n - new)]))
                top = float(x.abs().max())
                out["k_scale"][at] = top / 448.0 if top > 0 else 1.0
                out["k"][at, :len(x)] = _nearest_e4m3(x / out["k_scale"][at])
    else:
        out["k"][blk, slot] = k
    return out


def _exact_read(s):
    c = s["case"]
    d, ks, kvs = c["d"], [], []
    for b, n in enumerate(s["n"]):
        at = s["table"][b, :(n + BLOCK - 1) // BLOCK].long()
        kv = s["kv"][at]
        if c["kv"] == "fp8":
            sc = kv[..., d:d + 4 * ((d + 127) // 128)].contiguous().view(torch.float32).double()
            e = torch.arange(d, device="cuda") // 128
            kv = kv[..., :d].contiguous().view(torch.float8_e4m3fn).double() * sc[..., e]
        k = s["k"][at]
        if c["mode"] == "bf16_kfp8":
            k = k.view(torch.float8_e4m3fn).double() * s["k_scale"][at].double()[:, None, None]
        elif c["mode"] == "mxfp8":
            x = torch.pow(2.0, s["k_scale"][at].double() - 127)
            k = (k.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32)) * x[..., None]).flatten(-2)
        ks.append(k.double().flatten(0, 1)[:n])
        kvs.append(kv.double().flatten(0, 1)[:n])
    return [torch.cat(ks), torch.cat(kvs)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        rot = case["rot"]
        return [_turned(s["x"][..., 128:], s["pos"], s["freq"], case["layout"], s["scale"], case["transpose"]),
                _turned(s["x_I"][..., :rot], s["pos"], s["freq"], case["layout_I"], s["scale"], case["transpose"])]
    return {"append": _exact_append, "read": _exact_read, "attn": _exact_attn}[case["op"]](s)
