"""The operators of grouped-head layers in a model's decode step: the append of new keys and values into
a paged cache of 8-bit codes (one scale per 64-token block and key head), attention over that cache, the
attention weight that each cached position receives, and the eviction of light positions.

``run`` makes one pass of an operator: in plain torch where ``own`` is false, through the library's
entry points where it is true. ``exact`` computes the same outputs in 64 bits from the definitions.

Shapes: 32 / 8 and 64 / 8 heads of 128 are the prompt attention's grouped heads, 8 / 2 heads the tiny
fp32 decode's; batches of 32 with 16K to 32K positions, one sequence of 1M positions and serving batches
of mixed lengths are the decode configurations'.
"""
import math
import random

import torch

own = False

BLOCK = 64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------ cases

def listed():
    wide = dict(type="bf16", H=64, H_kv=8, d_qk=128, d_v=128)
    mid = dict(type="bf16", H=32, H_kv=8, d_qk=128, d_v=128)
    tiny = dict(type="f32", H=8, H_kv=2, d_qk=128, d_v=128)
    return [
        # decode step: one new token for each of 32 sequences
        dict(name="append decode 32", op="append", **mid, B=32, new=1, ragged=False, most=4096, lens=1),
        # a prompt's keys and values, two sequences of 4096 new tokens behind cached ones
        dict(name="append prompt 2x4096", op="append", **mid, B=2, new=4096, ragged=False, most=6000, lens=2),
        # chunks of different lengths in fp32, of which some continue a block
        dict(name="append fp32 ragged", op="append", **tiny, B=7, new=300, ragged=True, most=700, lens=3),
        # the smallest decode step: one sequence, fp32, where latency counts
        dict(name="attn fp32 one of 2048", op="attn", **tiny, B=1, new=1, least=2048, most=2048, weights=False, lens=4),
        # the decode batch of 32 sequences of 16K to 32K positions
        dict(name="attn decode 32 x 16K-32K", op="attn", **wide, B=32, new=1, least=16384, most=32768, weights=False, lens=5),
        # one sequence of 1M positions: the largest case
        dict(name="attn one of 1M", op="attn", **mid, B=1, new=1, least=1048576, most=1048576, weights=False, lens=6),
        # four drafted tokens for each of 16 sequences of mixed lengths
        dict(name="attn drafts 16 x 4", op="attn", **wide, B=16, new=4, least=4, most=16001, weights=False, lens=7),
        # a decode batch that keeps count of the weight every position receives
        dict(name="weights decode 32 x 8K", op="attn", **mid, B=32, new=1, least=1000, most=8191, weights=True, lens=8),
        # the same for a few short fp32 sequences
        dict(name="weights fp32 short", op="attn", **tiny, B=5, new=1, least=1, most=600, weights=True, lens=9),
        # a serving batch brought down to half of its positions
        dict(name="evict 8 x 16K to 8K", op="evict", **mid, B=8, least=12000, most=16384, keep=8192, sink=4, recent=1024, lens=10),
        # one long context cut to a quarter
        dict(name="evict 128K to 32K", op="evict", **mid, B=1, least=131072, most=131072, keep=32768, sink=16, recent=4096, lens=11),
        # many short sequences, some of which stay whole
        dict(name="evict 33 short", op="evict", **tiny, B=33, least=1, most=1000, keep=300, sink=1, recent=37, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "evict"])
    H, H_kv = rng.choice([(32, 8), (64, 8), (8, 2), (8, 8), (7, 1), (12, 4), (24, 8), (64, 1), (10, 2), (48, 16)])
    d_qk, d_v = rng.choice([(128, 128), (128, 128), (128, 128), (64, 64), (96, 96), (192, 128), (256, 256), (80, 48)])
    case = dict(op=op, type=rng.choice(["bf16", "bf16", "f32"]), H=H, H_kv=H_kv, d_qk=d_qk, d_v=d_v, lens=rng.randrange(1 << 20))
    if op == "append":
        new = rng.choice([1, _log(rng, 2, 4096)])
        return dict(case, B=_log(rng, 1, 64) if new == 1 else rng.randint(1, 3), new=new, ragged=rng.random() < 0.5,
                    most=new + _log(rng, 1, 4096))
    if op == "evict":
        B, most = _log(rng, 1, 40), _log(rng, 2, 65536)
        while B * most * H_kv * (d_qk + d_v) > (1 << 29):
            B = max(1, B - 1) if B > 1 else B
            most = max(2, most * 3 // 4)
        keep = max(1, int(most * rng.uniform(0.1, 0.9)))
        sink = rng.choice([0, 1, 4, rng.randint(0, keep)])
        sink = min(sink, keep)
        return dict(case, B=B, least=rng.randint(1, most), most=most, keep=keep, sink=sink, recent=rng.randint(0, (keep - sink) // 2))
    B, most = _log(rng, 1, 64), _log(rng, 1, 65536)
    new = rng.choice([1, 1, 1, 2, rng.randint(2, 16)])
    while B * most * (H_kv * (d_qk + d_v) + 2 * new * H) > (1 << 30):
        B, most = max(1, B * 3 // 4), max(1, most * 3 // 4)
    return dict(case, B=B, new=new, least=rng.choice([0, 1, most]), most=most, weights=rng.random() < 0.35)


def lengths(case):
    """Cached positions of every sequence, the call's new tokens included: a part of the case."""
    r = random.Random(case["lens"])
    most, least = case["most"], case.get("least", case.get("new", 1))
    n = [most] + [r.randint(min(least, most), most) for _ in range(case["B"] - 1)]
    r.shuffle(n)
    return n


def news(case, n):
    """New tokens of every sequence: the case's number, or some up to it (no more than it has positions)."""
    r = random.Random(case["lens"] + 1)
    new = case.get("new", 1)
    return [min(r.randint(0, new), v) if case.get("ragged") else min(new, v) if case["op"] == "append" else new for v in n]


def starts(n):
    s = [0]
    for v in n:
        s.append(s[-1] + v)
    return s


# ----------------------------------------------------------------------------------------- inputs

def _tables(n, first, g):
    """Shuffled block tables for sequences of n positions over blocks first, first + 1, ...: (table, blocks)."""
    blocks = [(v + BLOCK - 1) // BLOCK for v in n]
    total, width = sum(blocks) + 2, max(1, max(blocks))
    perm = (first + torch.randperm(total, generator=g, device="cuda")).to(torch.int32)
    col = torch.arange(width, device="cuda")
    nb = torch.tensor(blocks, device="cuda")
    begin = torch.tensor(starts(blocks)[:-1], device="cuda")
    src = (begin[:, None] + col[None]).clamp(max=total - 1)
    return torch.where(col[None] < nb[:, None], perm[src], -1), total


def _cache(blocks, H_kv, d, g):
    """Quantised normal values: codes [blocks][H_kv][64][d], scales [blocks][H_kv]."""
    codes = torch.empty((blocks, H_kv, BLOCK, d), dtype=torch.uint8, device="cuda")
    scale = torch.empty((blocks, H_kv), dtype=torch.float32, device="cuda")
    for i in range(0, blocks, 4096):
        x = torch.randn((min(4096, blocks - i), H_kv, BLOCK, d), generator=g, device="cuda")
        scale[i:i + 4096] = s = x.abs().amax(dim=(2, 3)) / 448.0
        codes[i:i + 4096] = (x / s[..., None, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    B, H, H_kv, t = case["B"], case["H"], case["H_kv"], DTYPES[case["type"]]
    n = lengths(case)
    s = dict(case=case, n=n, seq_lens=ints(n))
    s["table"], blocks = _tables(n, 0, g)
    if case["op"] == "evict":
        keep = case["keep"]
        s["new_table"], more = _tables([min(v, keep) for v in n], blocks, g)
        blocks += more
    s["k"], s["k_scale"] = _cache(blocks, H_kv, case["d_qk"], g)
    s["v"], s["v_scale"] = _cache(blocks, H_kv, case["d_v"], g)
    s["blocks"] = blocks
    width = s["table"].shape[1] * BLOCK
    if case["op"] == "evict":
        s["weights"] = torch.randn((B, H_kv, width), generator=g, device="cuda").mul_(2.0).exp_()  # a heavy tail
        s["kept"] = torch.empty((B, H_kv, case["keep"]), dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.empty((B,), dtype=torch.int32, device="cuda")
        s["weights_out"] = torch.empty((B, H_kv, s["new_table"].shape[1] * BLOCK), device="cuda")
        s["scratch"] = torch.zeros(1024, dtype=torch.uint8, device="cuda")
        return s
    new = news(case, n)
    s["new"], s["cu"] = new, None if new == [1] * B else ints(starts(new))
    T = sum(new)
    if case["op"] == "append":
        # keys carry a few loud columns, values do not
        loud = 1.0 + 7.0 * (torch.rand(case["d_qk"], generator=g, device="cuda") < 0.05)
        s["k_new"] = (torch.randn((T, H_kv, case["d_qk"]), generator=g, device="cuda") * loud).to(t)
        s["v_new"] = torch.randn((T, H_kv, case["d_v"]), generator=g, device="cuda").to(t)
        s["scratch"] = torch.zeros(1024, dtype=torch.uint8, device="cuda")
        return s
    # heads from flat to peaked attention
    sharp = torch.exp2(3.0 * torch.rand((H, 1), generator=g, device="cuda") - 1.0)
    s["q"] = (torch.randn((T, H, case["d_qk"]), generator=g, device="cuda") * sharp).to(t)
    s["sm_scale"] = case["d_qk"] ** -0.5
    s["weights"] = s["weights_out"] = None
    if case["weights"]:
        s["weights"] = torch.rand((B, H_kv, width), generator=g, device="cuda")
        s["weights_out"] = torch.zeros((B, H_kv, width), device="cuda")
    scores = (T * (H // H_kv) + BLOCK * B) * H_kv * (width + 128) if case["weights"] else 0
    s["scratch"] = torch.empty((64 << 20) + 4 * scores, dtype=torch.uint8, device="cuda")  # kept from step to step
    s["scratch"][:1024] = 0
    return s


# ------------------------------------------------------------------------------------- plain forms

def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes, scale):
    return codes.view(torch.float8_e4m3fn).float().mul_(scale)


def _unit(amax):
    """The scale that takes amax to the largest code."""
    return torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))


def _written(s):
    """The caches as outputs: codes as the values they stand for."""
    return {"k": s["k"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"], "v": s["v"].view(torch.float8_e4m3fn),
            "v_scale": s["v_scale"]}


def _rows(s):
    """Sequence and position of every new token."""
    B, dev = s["case"]["B"], s["seq_lens"].device
    cu = torch.arange(B + 1, device=dev) if s["cu"] is None else s["cu"].long()
    r = torch.arange(sum(s["new"]), device=dev)
    seq = torch.searchsorted(cu[1:].contiguous(), r, right=True)
    return seq, s["seq_lens"].long()[seq] - (cu[seq + 1] - cu[seq]) + r - cu[seq]


def _append(cache, scale, x, blk, slot):
    """Rows x [T][H_kv][d] into (blk, slot), every block and head against its own scale."""
    x = x.float()
    nb, H_kv = scale.shape
    first = torch.full((nb,), BLOCK, dtype=torch.int64, device=x.device).scatter_reduce_(0, blk, slot, "amin")
    amax = torch.zeros_like(scale).scatter_reduce_(0, blk[:, None].expand(-1, H_kv), x.abs().amax(dim=2), "amax")
    at = torch.nonzero(first < BLOCK)[:, 0]  # the blocks that get tokens
    f, a, old = first[at], amax[at], scale[at]
    new = torch.where(f[:, None] == 0, _unit(a), torch.maximum(old, a / 448.0))
    codes = cache[at]
    again = (new > old)[..., None, None] & (torch.arange(BLOCK, device=x.device) < f[:, None])[:, None, :, None]
    again = _e4m3(_values(codes, old[..., None, None]) / new[..., None, None]).where(again, codes)
    scale[at] = new
    cache[at] = again
    cache[blk, :, slot] = _e4m3(x / scale[blk][..., None])


def _plain_append(s):
    seq, pos = _rows(s)
    blk, slot = s["table"][seq, pos // BLOCK].long(), pos % BLOCK
    _append(s["k"], s["k_scale"], s["k_new"], blk, slot)
    _append(s["v"], s["v_scale"], s["v_new"], blk, slot)
    return _written(s)


def _gathered(cache, scale, table):
    """The sequences' rows in fp32, [B][H_kv][positions][d]."""
    t = table.clamp(min=0).long()
    x = _values(cache[t], scale[t][..., None, None])
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attn(s):
    c = s["case"]
    B, H, H_kv = c["B"], c["H"], c["H_kv"]
    G, most, dev = H // H_kv, max(1, max(s["new"])), s["q"].device
    seq, pos = _rows(s)
    cu = torch.arange(B, device=dev) if s["cu"] is None else s["cu"].long()[:-1]
    i = torch.arange(len(seq), device=dev) - cu[seq]
    q = torch.zeros((B, most, H, c["d_qk"]), device=dev)
    q[seq, i] = s["q"].float() * s["sm_scale"]
    sees = torch.full((B, most), -1, dtype=torch.int64, device=dev)
    sees[seq, i] = pos
    q = q.view(B, most, H_kv, G, -1).permute(0, 2, 3, 1, 4).reshape(B, H_kv, G * most, -1)
    k = _gathered(s["k"], s["k_scale"], s["table"])
    z = q @ k.transpose(-1, -2)
    del k
    hidden = torch.arange(z.shape[-1], device=dev) > sees[:, :, None]
    z.view(B, H_kv, G, most, -1).masked_fill_(hidden[:, None, None], -math.inf)
    m = z.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = z.sub_(m).exp_()
    l = p.sum(dim=-1, keepdim=True)
    lse = (m + l.log()).view(B, H_kv, G, most).permute(0, 3, 1, 2).reshape(B, most, H)[seq, i]
    p.div_(torch.where(l > 0, l, torch.ones_like(l)))
    if s["weights"] is not None:
        live = torch.arange(p.shape[-1], device=dev) < s["seq_lens"][:, None]
        s["weights_out"].copy_(torch.where(live[:, None], s["weights"] + p.sum(dim=2), s["weights_out"]))
    o = p @ _gathered(s["v"], s["v_scale"], s["table"])
    o = o.view(B, H_kv, G, most, -1).permute(0, 3, 1, 2, 4).reshape(B, most, H, -1)[seq, i]
    out = {"out": o.to(s["q"].dtype), "lse": lse}
    if s["weights"] is not None:
        out["weights"] = s["weights_out"]
    return out


def _move(cache, scale, kept, n, s):
    """Rows `kept` of every sequence and head into the new blocks."""
    keep, dev = s["case"]["keep"], kept.device
    B, H_kv, _ = kept.shape
    h = torch.arange(H_kv, device=dev)[None, :, None]
    blk = s["table"].long()[torch.arange(B, device=dev)[:, None, None], kept.clamp(min=0) // BLOCK]
    codes, old = cache[blk, h, kept % BLOCK], scale[blk, h]
    live = kept >= 0
    x = torch.where(live[..., None], _values(codes, old[..., None]), 0.0)
    nb = s["new_table"].shape[1]
    pad = lambda t: torch.nn.functional.pad(t, (0, 0, 0, nb * BLOCK - keep) if t.dim() == 4 else (0, nb * BLOCK - keep))  # noqa: E731
    x, codes, live, old = (pad(t) if nb * BLOCK >= keep else t[:, :, :nb * BLOCK] for t in (x, codes, live, old))
    x, codes = x.unflatten(2, (nb, BLOCK)), codes.unflatten(2, (nb, BLOCK))
    live, old = live.unflatten(2, (nb, BLOCK)), old.unflatten(2, (nb, BLOCK))
    whole = (n <= keep)[:, None, None]
    new = torch.where(whole, old[..., 0], _unit(x.abs().amax(dim=(3, 4))))
    codes = torch.where(whole[..., None, None], codes, _e4m3(x / new[..., None, None]))
    at = s["new_table"].long()
    b, h, j, r = torch.nonzero(live, as_tuple=True)
    cache[at[b, j], h, r] = codes[b, h, j, r]
    b, h, j = torch.nonzero(live[..., 0], as_tuple=True)
    scale[at[b, j], h] = new[b, h, j]


def _plain_evict(s):
    c, w = s["case"], s["weights"]
    keep, sink, recent = c["keep"], c["sink"], c["recent"]
    n = s["seq_lens"].long()
    pos = torch.arange(w.shape[2], device=w.device)
    held = (pos < sink) | (pos >= (n - recent)[:, None])
    rank = torch.where(pos >= n[:, None], 0, torch.where(held, 2, 1))[:, None].expand_as(w)
    order = torch.sort(w, dim=2, descending=True, stable=True).indices  # ties stay in order of position
    order = order.gather(2, torch.sort(rank.gather(2, order), dim=2, descending=True, stable=True).indices)
    short = max(0, keep - w.shape[2])
    kept = order[:, :, :keep]
    kept = torch.where(kept < n[:, None, None], kept, w.shape[2])
    kept = torch.nn.functional.pad(torch.sort(kept, dim=2).values, (0, short), value=w.shape[2])
    kept = torch.where(kept < w.shape[2], kept, -1)
    s["kept"].copy_(kept)
    s["new_lens"].copy_(n.clamp(max=keep))
    got = torch.where(kept >= 0, w.gather(2, kept.clamp(min=0)), 0.0)[:, :, :s["weights_out"].shape[2]]
    s["weights_out"].zero_()[:, :, :got.shape[2]] = got
    _move(s["k"], s["k_scale"], kept, n, s)
    _move(s["v"], s["v_scale"], kept, n, s)
    return {"kept": s["kept"], "lens": s["new_lens"], "weights": s["weights_out"], **_written(s)}


# ------------------------------------------------------------------------------- the library's calls

def _dims(s):
    import indexer_top_sparse_paged_gb300 as dsa
    c = s["case"]
    return dsa.grouped_dims(c["type"], c["B"], s["table"].shape[1], s["blocks"], c["H"], c["H_kv"], c["d_qk"], c["d_v"])


def _own_append(s):
    import indexer_top_sparse_paged_gb300 as dsa
    dsa.grouped_append(_dims(s), s["k_new"], s["v_new"], s["table"], s["seq_lens"], s["k"], s["k_scale"], s["v"], s["v_scale"],
                       s["cu"], ws=s["scratch"])
    return _written(s)


def _own_attn(s):
    import indexer_top_sparse_paged_gb300 as dsa
    out, lse = dsa.grouped_attn(_dims(s), s["q"], s["k"], s["k_scale"], s["v"], s["v_scale"], s["table"], s["seq_lens"],
                                s["sm_scale"], s["cu"], weights=s["weights"], weights_out=s["weights_out"], ws=s["scratch"])
    return {"out": out, "lse": lse} if s["weights"] is None else {"out": out, "lse": lse, "weights": s["weights_out"]}


def _own_evict(s):
    import indexer_top_sparse_paged_gb300 as dsa
    c = s["case"]
    dsa.grouped_evict(_dims(s), s["weights"], c["keep"], s["table"], s["seq_lens"], s["new_table"], s["k"], s["k_scale"], s["v"],
                      s["v_scale"], sink=c["sink"], recent=c["recent"], kept=s["kept"], new_lens=s["new_lens"],
                      weights_out=s["weights_out"], ws=s["scratch"])
    return {"kept": s["kept"], "lens": s["new_lens"], "weights": s["weights_out"], **_written(s)}


def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "attn": _own_attn, "evict": _own_evict}[op](s)
    return {"append": _plain_append, "attn": _plain_attn, "evict": _plain_evict}[op](s)


# --------------------------------------------------------------------------------- what a pass needs

def work(case):
    n = lengths(case)
    H, H_kv, d = case["H"], case["H_kv"], case["d_qk"] + case["d_v"]
    e = 4 if case["type"] == "f32" else 2
    if case["op"] == "append":
        T = max(1, sum(news(case, n)))
        return {"bytes": T * H_kv * d * (e + 1), "flops": 2 * T * H_kv * d}
    if case["op"] == "evict":
        kept = sum(min(v, case["keep"]) for v in n)
        return {"bytes": H_kv * (4 * sum(n) + kept * (2 * d + 8)), "flops": H_kv * (sum(n) + 2 * kept * d)}
    new = news(case, n)
    pairs = sum(max(0, v - m + i + 1) for v, m in zip(n, new) for i in range(m))
    T = max(1, sum(new))
    return {"bytes": sum(n) * H_kv * (d + (8 if case["weights"] else 0)) + T * H * (d * e + 4), "flops": 2 * max(1, pairs) * H * d}


# ------------------------------------------------------------------------------------------ 64 bits

def _nearest_e4m3(x):
    """The e4m3 value nearest to x (ties to the even code), saturating, by search in the ordered table."""
    table = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(table, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - table[lo], table[hi] - a
    pick = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return table[pick] * torch.where(x < 0, -1.0, 1.0)


def _exact_append(s):
    out = {name: v.double() for name, v in _written(s).items()}
    for name in ("k", "v"):
        codes, scale, x, r = out[name], out[name + "_scale"], s[name + "_new"].double(), 0
        for b, (n, m) in enumerate(zip(s["n"], s["new"])):
            p = n - m
            while p < n:  # block by block
                at, lo = int(s["table"][b, p // BLOCK]), p % BLOCK
                k = min(BLOCK - lo, n - p)
                rows = x[r:r + k].transpose(0, 1)
                top = rows.abs().amax(dim=(1, 2)) / 448.0
                unit = torch.where(top > 0, top, 1.0)
                if lo:
                    unit = torch.maximum(scale[at], top)
                    ratio = (scale[at] / unit)[:, None, None]
                    codes[at, :, :lo] = torch.where(ratio < 1, _nearest_e4m3(codes[at, :, :lo] * ratio), codes[at, :, :lo])
                codes[at, :, lo:lo + k] = _nearest_e4m3(rows / unit[:, None, None])
                scale[at] = unit
                p, r = p + k, r + k
    return out


def _dense(s, name, b, h):
    n = s["n"][b]
    at = s["table"][b, :(n + BLOCK - 1) // BLOCK].long()
    x = s[name][at, h].view(torch.float8_e4m3fn).double() * s[name + "_scale"][at, h].double()[:, None, None]
    return x.flatten(0, 1)[:n]


def _exact_attn(s):
    c, dev = s["case"], s["q"].device
    G, T = c["H"] // c["H_kv"], sum(s["new"])
    out = torch.zeros((T, c["H"], c["d_v"]), dtype=torch.float64, device=dev)
    lse = torch.full((T, c["H"]), -math.inf, dtype=torch.float64, device=dev)
    weights = s["weights_out"].double() if s["weights"] is not None else None
    r = 0
    for b, (n, m) in enumerate(zip(s["n"], s["new"])):
        for h in range(c["H_kv"] if n else 0):
            k, v = _dense(s, "k", b, h), _dense(s, "v", b, h)
            total = torch.zeros(n, dtype=torch.float64, device=dev)
            for i in range(m):
                e = n - m + i + 1
                if e > 0:
                    z = s["q"][r + i, h * G:h * G + G].double() @ k[:e].T * s["sm_scale"]
                    lse[r + i, h * G:h * G + G] = torch.logsumexp(z, dim=1)
                    p = torch.softmax(z, dim=1)
                    out[r + i, h * G:h * G + G] = p @ v[:e]
                    total[:e] += p.sum(0)
            if weights is not None:
                weights[b, h, :n] = s["weights"][b, h, :n].double() + total
        r += m
    return {"out": out, "lse": lse} if weights is None else {"out": out, "lse": lse, "weights": weights}


def _exact_evict(s):
    c = s["case"]
    keep, sink, recent = c["keep"], c["sink"], c["recent"]
    kept, lens = torch.full_like(s["kept"], -1), torch.zeros_like(s["new_lens"])
    weights = torch.zeros_like(s["weights_out"], dtype=torch.float64)
    out = {name: v.double() for name, v in _written(s).items()}
    for b, n in enumerate(s["n"]):
        m = min(n, keep)
        lens[b] = m
        for h in range(c["H_kv"] if n else 0):
            w = s["weights"][b, h, :n].double()
            at = torch.arange(n, device=w.device)
            if n > keep:
                w = w.clone()
                w[:sink], w[n - recent:] = math.inf, math.inf
                at = torch.sort(torch.argsort(w, descending=True, stable=True)[:keep]).values
            kept[b, h, :m] = at
            weights[b, h, :m] = s["weights"][b, h, at].double()
            for name in ("k", "v"):
                old = s["table"][b].long()[at // BLOCK]
                code = s[name][old, h, at % BLOCK].view(torch.float8_e4m3fn).double()
                x = code * s[name + "_scale"][old, h].double()[:, None]
                for j in range(0, m, BLOCK):
                    to, rows = int(s["new_table"][b, j // BLOCK]), x[j:j + BLOCK]
                    top = rows.abs().max()
                    unit = s[name + "_scale"][old[j], h].double() if n <= keep else torch.where(top > 0, top / 448.0, 1.0)
                    out[name][to, h, :len(rows)] = code[j:j + BLOCK] if n <= keep else _nearest_e4m3(rows / unit)
                    out[name + "_scale"][to, h] = unit
    return {"kept": kept, "lens": lens, "weights": weights, **out}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "append" and sum(s["n"]) * case["H_kv"] > (1 << 24):
        return None
    return {"append": _exact_append, "attn": _exact_attn, "evict": _exact_evict}[case["op"]](s)
