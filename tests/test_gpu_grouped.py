"""The grouped-head cache in 8 bits (dsa_grouped_append, dsa_grouped_attn, dsa_grouped_evict) against the definitions in
64 bits: lengths from none to many tiles, drafts, grouped heads, widths, strided views, queries without positions, codes
of NaN in unused slots, invalid blocks and sequences, weights, ties, graphs and streams."""
import math

import pytest
import torch

import indexer_top_sparse_paged_gb300 as dsa

pytestmark = pytest.mark.gpu
ACT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAN_CODE = 0x7F


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts(n):
    return ints([0] + torch.tensor(n, dtype=torch.int64).cumsum(0).tolist())


def value(codes):
    return codes.view(torch.float8_e4m3fn).double()


class Cache:
    """Caches of sequences of `lens` positions (room for `room`) in shuffled blocks; unused slots and blocks hold NaN codes."""

    def __init__(self, lens, H, H_kv, d_qk, d_v, type="bf16", seed=0, room=None, spread=1.0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.H, self.H_kv, self.d_qk, self.d_v, self.type = list(lens), H, H_kv, d_qk, d_v, type
        room = room or [max(1, n) for n in lens]
        need = [(max(n, r) + 63) // 64 for n, r in zip(lens, room)]
        self.blocks, self.width = sum(need) + 3, max(need) + 1
        perm = torch.randperm(self.blocks, generator=self.g, device="cuda").to(torch.int32)
        self.table = torch.full((len(lens), self.width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.free = perm[at:]
        make = lambda d: torch.full((self.blocks, H_kv, 64, d), NAN_CODE, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.k, self.v = make(d_qk), make(d_v)
        self.ks, self.vs = (torch.full((self.blocks, H_kv), float("nan"), device="cuda") for _ in range(2))
        for cache, scale, d in ((self.k, self.ks, d_qk), (self.v, self.vs, d_v)):
            for b, n in enumerate(self.lens):
                for j in range((n + 63) // 64):
                    m, blk = min(64, n - 64 * j), int(self.table[b, j])
                    x = torch.randn((H_kv, m, d), generator=self.g, device="cuda")
                    scale[blk] = x.abs().amax(dim=(1, 2)) / 448 * spread ** (j % 5 - 2)
                    cache[blk, :, :m] = (x * 448 / x.abs().amax(dim=(1, 2), keepdim=True)).to(torch.float8_e4m3fn).view(torch.uint8)
        self.seq_lens = ints(self.lens)

    def dims(self):
        return dsa.grouped_dims(self.type, len(self.lens), self.width, self.blocks, self.H, self.H_kv, self.d_qk, self.d_v)

    def args(self):
        return self.k, self.ks, self.v, self.vs, self.table, self.seq_lens

    def rows(self, b, h):
        """(k, v) of sequence b and key head h in fp64, and which positions are in valid blocks."""
        n = self.lens[b]
        at = self.table[b, :(n + 63) // 64].long()
        ok = (at >= 0) & (at < self.blocks)
        at = at.clamp(0, self.blocks - 1)
        k = (value(self.k[at, h]) * self.ks[at, h].double()[:, None, None]).flatten(0, 1)[:n]
        v = (value(self.v[at, h]) * self.vs[at, h].double()[:, None, None]).flatten(0, 1)[:n]
        ok = ok.repeat_interleave(64)[:n]
        return torch.where(ok[:, None], k, 0.0), torch.where(ok[:, None], v, 0.0), ok

    def queries(self, T, sharp=1.0):
        return (sharp * torch.randn((T, self.H, self.d_qk), generator=self.g, device="cuda")).to(ACT[self.type])


def check(c, q, new, got, scale, weights=None, weights_out=None):
    """(out, lse) and the weights of the queries q against softmax attention in 64 bits."""
    out, lse = got
    bf16 = c.type == "bf16"
    G, t0 = c.H // c.H_kv, 0
    u = 2.0 ** -24
    for b, (n, m) in enumerate(zip(c.lens, new)):
        for h in range(c.H_kv):
            k, v, ok = c.rows(b, h)
            w = torch.zeros(n, dtype=torch.float64, device="cuda")
            w_tol = torch.zeros_like(w)
            for i in range(m):
                Q = q[t0 + i, h * G:h * G + G].double()
                seen = (torch.arange(n, device="cuda") <= n - m + i) & ok
                z = (Q @ k.T * scale).masked_fill(~seen, -math.inf)
                e = torch.logsumexp(z, -1)
                o_got, e_got = out[t0 + i, h * G:h * G + G].double(), lse[t0 + i, h * G:h * G + G].double()
                if not seen.any():
                    assert not o_got.any() and bool((e_got == -math.inf).all())
                    continue
                p = torch.exp(z - e[:, None])
                # A logit: the products and their fp32 sum round d + 2 times, and the factor to powers of two and the
                # subtraction twice more. A bf16 query is split into two e4m3 parts, the second in units of 1/16: elements that
                # are normal in the first part are exact (8 bits), smaller ones are off by half a step of the second, 2^-10 / 16,
                # where the largest element stands above 224: 2^-14 / 224 < 2^-21 of it. fp32 ones, in six parts: less.
                ka = k.abs()
                z_tol = ((c.d_qk + 4) * u * (Q.abs() @ ka.T) + 2.0 ** -21 * Q.abs().amax(-1, keepdim=True) * ka.sum(-1)) * scale
                z_tol = torch.where(seen, z_tol, 0.0).amax(-1) + 2.0 ** -22 * (1 + z[:, seen].abs().amax(-1))
                # A weight: twice that, 2^-22 of the exponential, in bf16 2^-10 for its fp16 value and the parts of 4 bits it is
                # split into (2^-11 each), and 2^-26 of the largest weight absolutely; sums add one rounding a position.
                p_rel = 2 * z_tol + 2.0 ** -21 + (2.0 ** -10 if bf16 else 0.0) + (n + 8) * u
                mag = p @ v.abs() + 2.0 ** -26 * p.amax(-1, keepdim=True) * v[ok].abs().sum(0) * (1.0 if bf16 else 2.0 ** -10)
                o = p @ v
                tol = p_rel[:, None] * mag * 1.01 + (2.0 ** -8 if bf16 else 2.0 ** -22) * o.abs() * 1.01 + 1e-30
                tol = tol + 2.0 ** -26 * p.amax(-1, keepdim=True) * v[ok].abs().sum(0) * (1.01 if bf16 else 2.0 ** -10)
                err = (o_got - o).abs()
                assert bool((err <= tol).all()), (b, h, i, float((err - tol).max()), float(err.max()))
                e_tol = z_tol + (n + 8) * u + 2.0 ** -22 * (1 + e.abs())
                assert bool(((e_got - e).abs() <= e_tol).all()), (b, h, i, float(((e_got - e).abs() - e_tol).max()))
                w += p.sum(0)
                w_tol += ((2 * z_tol + e_tol + 2.0 ** -20)[:, None] * p).sum(0)
            if weights_out is not None:
                old = torch.zeros_like(w) if weights is None else weights[b, h, :n].double()
                err = (weights_out[b, h, :n].double() - old - w).abs()
                w_tol = w_tol + (m * G + 2) * u * (w + old.abs()) + 1e-30
                assert bool((err <= w_tol).all()), (b, h, float((err - w_tol).max()))
        t0 += m


def attend(c, q, new, scale, faults=0, **kw):
    ws = dsa.grouped_workspace(c.dims(), q.shape[0], weights=kw.get("weights_out") is not None or kw.get("weights") is not None)
    cu = None if new == [1] * len(c.lens) and q.shape[0] == len(c.lens) else starts(new)
    got = dsa.grouped_attn(c.dims(), q, *c.args(), scale, cu, ws=ws, **kw)
    assert dsa.read_error(ws) == faults
    return got


LENS = [([1], [1]), ([64], [1]), ([128, 129, 127], [1, 1, 1]), ([0, 5, 0, 700], [1, 1, 1, 1]), ([65, 1, 2048, 63], [3, 1, 2, 5]),
        ([300, 7, 40], [0, 4, 1]), ([3, 0, 1], [5, 2, 1]), ([5000], [1]), ([130, 2000], [16, 9])]


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("lens,new", LENS)
def test_lengths_and_drafts(type, lens, new):
    c = Cache(lens, 8, 2, 128, 128, type, seed=len(lens))
    q = c.queries(sum(new))
    check(c, q, new, attend(c, q, new, 128 ** -0.5), 128 ** -0.5)


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("H,H_kv", [(1, 1), (7, 1), (12, 4), (6, 6), (64, 8), (130, 1), (48, 2), (10, 2), (33, 1)])
def test_grouped_heads(type, H, H_kv):
    lens, new = [300, 70, 1], [1, 3, 1]
    c = Cache(lens, H, H_kv, 64, 64, type, seed=H)
    q = c.queries(sum(new))
    check(c, q, new, attend(c, q, new, 0.125), 0.125)


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("d_qk,d_v", [(192, 128), (16, 16), (80, 48), (96, 96), (64, 128), (128, 64), (256, 256), (208, 144), (16, 256), (240, 16)])
def test_widths(type, d_qk, d_v):
    lens, new = [150, 900], [2, 1]
    c = Cache(lens, 8, 2, d_qk, d_v, type, seed=d_qk + d_v)
    q = c.queries(sum(new))
    check(c, q, new, attend(c, q, new, d_qk ** -0.5), d_qk ** -0.5)


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_many_sequences_and_long_ones(type):
    """More sequences than a CTA has threads, most of them short or empty; then few long ones whose positions are split."""
    lens = [(i * 37) % 200 if i % 3 else 0 for i in range(700)]
    c = Cache(lens, 4, 2, 32, 32, type, seed=1)
    q = c.queries(700)
    check(c, q, [1] * 700, attend(c, q, [1] * 700, 0.2), 0.2)
    c = Cache([40000, 129, 7000], 16, 2, 64, 64, type, seed=2)
    q = c.queries(4)
    check(c, q, [1, 2, 1], attend(c, q, [1, 2, 1], 0.125), 0.125)


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_large_and_growing_logits(type):
    """Logits that grow along the positions move every row's maximum in every tile; huge ones; equal ones; scales of the
    blocks that lie far apart."""
    c = Cache([1500], 4, 1, 64, 64, type, seed=3)
    for j in range(24):
        c.ks[int(c.table[0, j])] *= 0.2 + j
    for sharp in (1.0, 64.0, 0.0):
        q = c.queries(1, sharp)
        check(c, q, [1], attend(c, q, [1], 0.5), 0.5)
    for spread in (1e3, 1e-4):
        c = Cache([1500, 40], 4, 1, 64, 64, type, seed=4, spread=spread)
        c.ks.fill_(0.01)
        q = c.queries(2)
        check(c, q, [1, 1], attend(c, q, [1, 1], 0.125), 0.125)


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_one_heavy_position_among_many_light_ones(type):
    """Half of the weight on one position, the other half evenly on 30,000: light weights are not lost."""
    n = 30001
    c = Cache([n], 2, 1, 16, 16, type, seed=5)
    c.k[c.table[0, :469].long()] = 0
    c.k[int(c.table[0, 0]), 0, 3, 0] = 0x38  # 1.0
    c.ks.fill_(1.0)
    c.vs.fill_(1.0)
    c.v[c.table[0, :469].long()] = 0x38
    c.v[int(c.table[0, 0]), 0, 3] = 0
    q = torch.zeros((1, 2, 16), dtype=ACT[type], device="cuda")
    q[..., 0] = math.log(n - 1)
    out, lse = attend(c, q, [1], 1.0)
    check(c, q, [1], (out, lse), 1.0)
    assert abs(float(out.float().mean()) - 0.5) < 0.01


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_strided_queries_and_rows_left_alone(type):
    c = Cache([300, 64, 5], 8, 2, 64, 32, type, seed=6)
    new = [2, 0, 1]
    wide = torch.full((9, 8, 192), float("nan"), dtype=ACT[type], device="cuda")
    q = wide[..., 64:128]
    q[:3] = c.queries(3)
    out = torch.full((9, 8, 32), 3.0, dtype=ACT[type], device="cuda")
    lse = torch.full((9, 8), 4.0, device="cuda")
    ws = dsa.grouped_workspace(c.dims(), 9)
    dsa.grouped_attn(c.dims(), q, *c.args(), 0.125, starts(new), ws=ws, out=out, lse=lse)
    assert dsa.read_error(ws) == 0
    check(c, q, new, (out, lse), 0.125)
    assert bool((out[3:] == 3.0).all()) and bool((lse[3:] == 4.0).all())
    q = c.queries(3).transpose(0, 1).contiguous().transpose(0, 1)  # heads outermost
    got = attend(c, q, new, 0.125)
    check(c, q, new, got, 0.125)
    q = c.queries(1)[:, :1].expand(3, 8, 64)  # one row for all
    check(c, q, new, attend(c, q, new, 0.125), 0.125)


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_queries_of_nan_and_infinity(type):
    c = Cache([200, 300, 0], 8, 2, 64, 64, type, seed=7)
    new = [2, 1, 1]
    q = c.queries(4)
    ref, ref_lse = attend(c, q, new, 0.125)
    q[0, 1, 3], q[2, 5, 0], q[3, 0, 0] = float("nan"), math.inf, float("nan")
    w = torch.zeros((3, 2, c.width * 64), device="cuda")
    out, lse = attend(c, q, new, 0.125, weights_out=w)
    bad = torch.zeros((4, 8), dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[2, 5] = True
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(out[~bad], ref[~bad]) and torch.equal(lse[~bad], ref_lse[~bad])
    assert w[0, 0, :199].isnan().all() and w[1, 1, :300].isnan().all()
    assert not w[0, 0, 199:].isnan().any() and not w[0, 1].isnan().any() and not w[1, 0].isnan().any() and not w[2].any()


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-30, 1e-10, 1e30, 3e38])
def test_queries_of_zeros_and_tiny_ones(type, scale):
    """Logits of 0, whatever the scale: the mean of what is seen, also where a tile holds positions that are not."""
    c = Cache([200, 3, 128], 8, 2, 32, 32, type, seed=18)
    new = [3, 1, 1]
    q = torch.zeros((5, 8, 32), dtype=ACT[type], device="cuda")
    if scale < 1:
        q[:, 1] = 1e-30  # a logit far below 2^-126
    w = torch.zeros((3, 2, c.width * 64), device="cuda")
    check(c, q, new, attend(c, q, new, scale, weights_out=w), scale, None, w)


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_invalid_blocks_and_sequences(type):
    c = Cache([700, 300, 130], 8, 2, 64, 64, type, seed=8)
    q = c.queries(3)
    c.table[0, 3], c.table[0, 10], c.table[1, 0] = -1, c.blocks, 1 << 30
    w = torch.rand((3, 2, c.width * 64), device="cuda")
    w0 = w.clone()
    got = attend(c, q, [1, 1, 1], 0.125, faults=1, weights=w)
    check(c, q, [1, 1, 1], got, 0.125, w0, w)
    c.table[2] = -1  # no valid block: no positions
    out, lse = attend(c, q, [1, 1, 1], 0.125, faults=1)
    assert not out[2].any() and bool((lse[2] == -math.inf).all())
    # sequences whose cu entries descend or leave the rows are skipped; lengths that leave the table have no positions
    c = Cache([200, 100, 64], 4, 1, 32, 32, type, seed=9)
    q = c.queries(4)
    ws = dsa.grouped_workspace(c.dims(), 4)
    for cu, live in (([0, 2, 1, 4], {0: (0, 2), 2: (1, 3)}), ([0, 1, 9, 4], {0: (0, 1)}), ([-1, 1, 2, 4], {1: (1, 1), 2: (2, 2)})):
        out, lse = torch.full((4, 4, 32), 7.0, dtype=ACT[type], device="cuda"), torch.full((4, 4), 7.0, device="cuda")
        dsa.grouped_attn(c.dims(), q, *c.args(), 0.2, ints(cu), ws=ws, out=out, lse=lse)
        assert dsa.read_error(ws) == 2, cu
        touched = torch.zeros(4, dtype=torch.bool)
        for b, (t0, m) in live.items():
            touched[t0:t0 + m] = True
        assert bool((lse[~touched] == 7.0).all()) and not (lse[touched] == 7.0).any()
    lens = c.seq_lens.clone()
    for bad in (-1, c.width * 64 + 1, (1 << 31) - 1):
        c.seq_lens = lens.clone()
        c.seq_lens[1] = bad
        out, lse = dsa.grouped_attn(c.dims(), q[:3], *c.args(), 0.2, ws=ws)
        assert dsa.read_error(ws) == 2 and not out[1].any() and bool((lse[1] == -math.inf).all())
        c.lens[1] = 0
        check(c, q, [1, 1, 1], (out, lse), 0.2)


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("H,H_kv,new", [(8, 2, [1, 1, 1, 1]), (64, 2, [3, 0, 2, 1]), (130, 1, [2, 1, 5, 1]), (4, 4, [9, 1, 1, 0])])
def test_weights(type, H, H_kv, new):
    """Added in place, into another tensor, and to nothing; positions behind a sequence's end stay as they were."""
    lens = [700, 300, 3, 0]
    c = Cache(lens, H, H_kv, 32, 48, type, seed=H)
    q = c.queries(sum(new), 2.0)
    base = torch.rand((4, H_kv, c.width * 64), device="cuda")
    w = base.clone()
    got = attend(c, q, new, 0.2, weights=w)
    check(c, q, new, got, 0.2, base, w)
    other = torch.full_like(base, 5.0)
    got2 = attend(c, q, new, 0.2, weights=base, weights_out=other)
    assert torch.equal(got[0], got2[0]) and torch.equal(got[1], got2[1])
    plain = attend(c, q, new, 0.2)
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
    fresh = torch.full_like(base, 5.0)
    attend(c, q, new, 0.2, weights_out=fresh)
    check(c, q, new, got, 0.2, None, fresh)
    for b, n in enumerate(lens):
        assert torch.equal(other[b, :, :n], w[b, :, :n])
        assert bool((other[b, :, n:] == 5.0).all()) and torch.equal(w[b, :, n:], base[b, :, n:]) and bool((fresh[b, :, n:] == 5.0).all())


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_repeats_graphs_and_streams(type):
    """The same bits call after call, from a captured graph with new inputs, from another stream, and from two streams at once."""
    c = Cache([9000, 64, 700, 0], 16, 2, 128, 128, type, seed=11)
    q = c.queries(4)
    w = torch.zeros((4, 2, c.width * 64), device="cuda")
    ws = dsa.grouped_workspace(c.dims(), 4, weights=True)
    run = lambda ws=ws, q=q, **kw: dsa.grouped_attn(c.dims(), q, *c.args(), 0.1, weights_out=w if ws is not None else None, ws=ws, **kw)  # noqa: E731
    ref = run()
    ref_w = w.clone()
    for _ in range(3):
        again = run()
        assert torch.equal(again[0], ref[0]) and torch.equal(again[1], ref[1]) and torch.equal(w, ref_w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(stream=side)
    side.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(w, ref_w)
    out, lse = torch.zeros_like(ref[0]), torch.zeros_like(ref[1])
    with torch.cuda.stream(side):
        run(out=out, lse=lse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run(out=out, lse=lse)
    torch.cuda.synchronize()
    q.copy_(c.queries(4))
    c.seq_lens.copy_(ints([8999, 1, 650, 0]))
    c.lens = [8999, 1, 650, 0]
    graph.replay()
    torch.cuda.synchronize()
    check(c, q, [1] * 4, (out, lse), 0.1, None, w)
    streams, spaces = [torch.cuda.Stream() for _ in range(2)], [dsa.grouped_workspace(c.dims(), 4) for _ in range(2)]
    torch.cuda.synchronize()
    both = [dsa.grouped_attn(c.dims(), q, *c.args(), 0.1, ws=s, stream=st) for _ in range(4) for s, st in zip(spaces, streams)]
    torch.cuda.synchronize()
    for o, e in both:
        assert torch.equal(o, out) and torch.equal(e, lse)


def test_a_larger_workspace_serves_smaller_calls():
    big = Cache([500] * 20, 16, 2, 64, 64, seed=12)
    ws = dsa.grouped_workspace(big.dims(), 60, weights=True)
    for B in (20, 3, 1):
        for m in (1, 3):
            c = Cache([500] * B, 16, 2, 64, 64, seed=B)
            q = c.queries(B * m)
            w = torch.zeros((B, 2, c.width * 64), device="cuda")
            got = dsa.grouped_attn(c.dims(), q, *c.args(), 0.1, starts([m] * B), weights=w, ws=ws)
            assert dsa.read_error(ws) == 0
            check(c, q, [m] * B, got, 0.1, None, w)


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("d_qk,d_v", [(128, 128), (192, 128), (64, 256), (256, 256), (16, 16)])
@pytest.mark.parametrize("G,new", [(5, 2), (8, 2), (16, 2), (32, 2), (40, 5)])
def test_rows_of_an_item_by_widths(type, d_qk, d_v, G, new):
    """Every number of rows that share a tile, with every number of 128-column chunks; items that CTAs cut and whole ones."""
    lens = [130, 3000]
    c = Cache(lens, G, 1, d_qk, d_v, type, seed=G + d_qk)
    q = c.queries(new + 1)
    w = torch.zeros((2, 1, c.width * 64), device="cuda")
    got = attend(c, q, [new, 1], d_qk ** -0.5, weights_out=w)
    check(c, q, [new, 1], got, d_qk ** -0.5, None, w)


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G,new", [(8, 1), (8, 2), (8, 4), (8, 8)])
def test_two_hundred_calls_in_a_row(type, d, G, new):
    """Every SM with several items, again and again: no wait runs out, and the last call has the bits of the first."""
    lens = [600 + 400 * b for b in range(10)]
    c = Cache(lens, 8 * G, 8, d, d, type, seed=d + new, room=[n + 8 for n in lens])
    q = c.queries(10 * new)
    ws = dsa.grouped_workspace(c.dims(), 10 * new)
    cu = starts([new] * 10)
    out, lse = dsa.grouped_attn(c.dims(), q, *c.args(), d ** -0.5, cu, ws=ws)
    first = out.clone(), lse.clone()
    for _ in range(200):
        dsa.grouped_attn(c.dims(), q, *c.args(), d ** -0.5, cu, out=out, lse=lse, ws=ws)
    assert dsa.read_error(ws) == 0
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G,new", [(8, 1), (8, 2), (8, 4), (8, 8)])
def test_two_hundred_calls_with_scales_apart(type, d, G, new):
    """Tiles whose blocks take turns among others: no wait runs out, and the last call has the bits of the first, which are right."""
    lens = [300 + 500 * b for b in range(10)]
    c = Cache(lens, 8 * G, 8, d, d, type, seed=d + new, room=[n + 8 for n in lens])
    c.vs *= torch.exp2(4.0 * torch.randn(c.vs.shape, generator=c.g, device="cuda"))
    q = c.queries(10 * new)
    w = torch.zeros((10, 8, c.width * 64), device="cuda")
    ws = dsa.grouped_workspace(c.dims(), 10 * new, weights=True)
    cu = starts([new] * 10)
    out, lse = dsa.grouped_attn(c.dims(), q, *c.args(), d ** -0.5, cu, weights_out=w, ws=ws)
    first = out.clone(), lse.clone(), w.clone()
    for _ in range(200):
        dsa.grouped_attn(c.dims(), q, *c.args(), d ** -0.5, cu, out=out, lse=lse, weights_out=w, ws=ws)
    assert dsa.read_error(ws) == 0
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1]) and torch.equal(w, first[2])
    check(c, q, [new] * 10, first[:2], d ** -0.5, None, w)


def test_weights_of_many_sequences():
    lens = [(i * 53) % 300 for i in range(300)]
    c = Cache(lens, 6, 2, 16, 16, seed=14)
    q = c.queries(300)
    w = torch.rand((300, 2, c.width * 64), device="cuda")
    base = w.clone()
    check(c, q, [1] * 300, attend(c, q, [1] * 300, 0.25, weights=w), 0.25, base, w)


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("lens,new,G", [([900, 0, 130], [10, 2, 3], 64), ([20000, 3000], [3, 5], 40), ([70], [1], 3), ([500] * 260, [3] * 260, 4)])
def test_weights_of_many_rows(type, lens, new, G):
    """Few position tiles, whose rows a CTA's warps share, and more tiles than CTAs; sequences past the first 256."""
    c = Cache(lens, G, 1, 32, 16, type, seed=G)
    q = c.queries(sum(new))
    w = torch.rand((len(lens), 1, c.width * 64), device="cuda")
    base = w.clone()
    check(c, q, new, attend(c, q, new, 0.2, weights=w, weights_out=w), 0.2, base, w)


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_logits_that_pass_the_maximum_by_a_little_and_by_much(type):
    """Maxima that rise from tile to tile by less than the slack of the weights' reference, by about it, and by far more; rows
    whose first tiles show them nothing (invalid blocks)."""
    for rise in (0.5, 2.5, 4.0, 6.0, 40.0):
        c = Cache([2100], 8, 1, 16, 16, type, seed=15)
        c.k[c.table[0, :33].long()] = 0
        c.k[c.table[0, :33].long(), 0, :, 0] = 0x38  # 1.0
        for j in range(33):
            c.ks[int(c.table[0, j])] = 0.01 + rise * (j // 2) * math.log(2.0)
        c.table[0, 0:5] = -1
        q = torch.zeros((1, 8, 16), dtype=ACT[type], device="cuda")
        q[0, :, 0] = torch.linspace(0.125, 1.0, 8, device="cuda").to(ACT[type])
        check(c, q, [1], attend(c, q, [1], 1.0, faults=1), 1.0)


def test_a_read_timeout_clears_what_a_call_left():
    c = Cache([700], 8, 2, 64, 64, seed=16)
    q = c.queries(1)
    ws = dsa.grouped_workspace(c.dims(), 1)
    ref = dsa.grouped_attn(c.dims(), q, *c.args(), 0.125, ws=ws)
    assert not ws[:256].any()  # arrivals are all taken back
    ws[16:200] = 3
    ws[:4] = torch.tensor([4, 0, 0, 0], dtype=torch.uint8)  # the timeout bit
    assert dsa.read_error(ws) == 4 and not ws[:256].any()
    got = dsa.grouped_attn(c.dims(), q, *c.args(), 0.125, ws=ws)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_one_workspace_for_the_librarys_calls():
    """A workspace that other calls of the library have written into serves this one."""
    c = Cache([9000, 300], 16, 2, 64, 64, seed=17)
    q = c.queries(2)
    p = torch.randn((300, 16, 64), device="cuda").bfloat16()
    kv = torch.randn((300, 2, 64), device="cuda").bfloat16()
    pd = dsa.prompt_dims(p, kv, kv, 1)
    n = max(dsa.grouped_workspace(c.dims(), 2).numel(), dsa.prompt_workspace(pd, 300).numel())
    ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = ws[-ws.data_ptr() % 256:][:n]
    ws[:256] = 0
    ref = attend(c, q, [1, 1], 0.125)
    for _ in range(3):
        dsa.prompt_attn(pd, p, kv, kv, starts([300]), starts([300]), 0.125, ws=ws)
        got = dsa.grouped_attn(c.dims(), q, *c.args(), 0.125, ws=ws)
        assert dsa.read_error(ws) == 0 and torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


# ------------------------------------------------------------------------------------------------ append

def expected_append(codes, scale, table, x, first):
    """The definition, block by block in fp32 on the CPU: rows x [n][H_kv][d] at positions first, first + 1, ... of the sequence
    whose blocks `table` names."""
    n, p = x.shape[0], first
    while p < first + n:
        blk, lo = int(table[p // 64]), p % 64
        m = min(64 - lo, first + n - p)
        rows = x[p - first:p - first + m].float().transpose(0, 1)
        top = rows.abs().amax(dim=(1, 2)) / 448.0
        if lo:
            old = scale[blk]
            new = torch.maximum(old, top)
            again = (codes[blk, :, :lo].view(torch.float8_e4m3fn).float() * old[:, None, None] / new[:, None, None])
            again = again.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            codes[blk, :, :lo] = torch.where((new > old)[:, None, None], again, codes[blk, :, :lo])
        else:
            new = torch.where(top > 0, top, 1.0)
        codes[blk, :, lo:lo + m] = (rows / new[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[blk] = new
        p += m


def same(a, b):
    return torch.equal(a.cpu().nan_to_num(nan=-7.0), b.cpu().nan_to_num(nan=-7.0)) if a.is_floating_point() else torch.equal(a.cpu(), b.cpu())


def append_and_check(c, new, spread=1.0, faults=0, strided=False):
    """Appends new[b] tokens to every sequence and compares all caches with the definition's, and new values with their codes."""
    T = sum(new)
    make = lambda d: (spread * torch.randn((T, c.H_kv, d + (32 if strided else 0)), generator=c.g, device="cuda")).to(ACT[c.type])[..., :d]  # noqa: E731
    k, v = make(c.d_qk), make(c.d_v)
    want = [t.cpu().clone() for t in (c.k, c.ks, c.v, c.vs)]
    t0, table = 0, c.table.cpu()
    for b, m in enumerate(new):
        expected_append(want[0], want[1], table[b], k[t0:t0 + m].cpu(), c.lens[b])
        expected_append(want[2], want[3], table[b], v[t0:t0 + m].cpu(), c.lens[b])
        c.lens[b] += m
        t0 += m
    c.seq_lens.copy_(ints(c.lens))
    ws = dsa.grouped_workspace(c.dims(), T)
    cu = None if new == [1] * len(c.lens) else starts(new)
    dsa.grouped_append(c.dims(), k, v, c.table, c.seq_lens, c.k, c.ks, c.v, c.vs, cu, ws=ws)
    assert dsa.read_error(ws) == faults
    for got, ref in zip((c.k, c.ks, c.v, c.vs), want):
        assert same(got, ref)
    t0 = 0
    for b, m in enumerate(new):  # half a step of a code's 3 bits, or of its smallest one, and the quotient's and scale's roundings
        pos = torch.arange(c.lens[b] - m, c.lens[b], device="cuda")
        blk = c.table[b].long()[pos // 64]
        for x, codes, scale in ((k, c.k, c.ks), (v, c.v, c.vs)):
            s = scale[blk].double()[..., None]
            y, x = value(codes[blk, :, pos % 64]) * s, x[t0:t0 + m].double()
            assert bool(((y - x).abs() <= torch.maximum(x.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -20)).all())
        t0 += m
    return k, v


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("lens,new", [([0], [1]), ([0, 63, 64, 130], [1, 1, 1, 1]), ([0, 10, 64, 0], [64, 200, 65, 0]), ([5], [1000]),
                                      ([1, 0, 100], [63, 0, 28])])
def test_append(type, lens, new):
    room = [n + m + 1 for n, m in zip(lens, new)]
    for H_kv, d_qk, d_v in ((2, 128, 128), (3, 16, 80), (1, 256, 192)):
        c = Cache(lens, 6, H_kv, d_qk, d_v, type, seed=len(new) + d_qk, room=room)
        append_and_check(c, new, strided=d_qk == 128)


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_append_step_by_step(type):
    """130 decode steps of rising, falling and zero values: scales grow within a block, never shrink, and start anew."""
    c = Cache([0, 60, 7], 4, 2, 32, 48, type, seed=21, room=[140, 200, 140])
    for i in range(130):
        append_and_check(c, [1, 1, 1], spread=[1.0, 0.1, 3.0, 0.0, 0.5, 8.0, 1e-3][i % 7] * 1.01 ** i)
    append_and_check(c, [0, 2, 0], spread=0.0)


def test_append_of_zeros_extremes_and_a_batch_of_many():
    c = Cache([0, 0], 2, 1, 16, 16, "f32", seed=22, room=[70, 70])
    append_and_check(c, [65, 3], spread=0.0)
    assert bool((c.ks[c.table[0, 0].long()] == 1.0).all())
    c = Cache([0, 40], 2, 1, 16, 16, "f32", seed=23, room=[70, 70])
    append_and_check(c, [65, 3], spread=1e30)
    c = Cache([i % 130 for i in range(600)], 2, 2, 16, 16, "bf16", seed=24, room=[140] * 600)
    append_and_check(c, [1] * 600)
    append_and_check(c, [i % 3 for i in range(600)])


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("d", [16, 128, 256])
def test_zeros_before_small_values(type, d):
    """Tokens of zeros (of either sign) leave a block without a scale: the first others set it. One head's zeros, or the keys'
    alone, do no more; a scale of 1 that values have stays."""
    c = Cache([0, 0, 0], 4, 2, d, d, type, seed=26, room=[140, 140, 140])
    ws = dsa.grouped_workspace(c.dims(), 8)

    def append(rows, new):
        k, v = (torch.stack(x).to(ACT[type]).cuda() for x in rows)
        c.lens = [n + m for n, m in zip(c.lens, new)]
        c.seq_lens.copy_(ints(c.lens))
        dsa.grouped_append(c.dims(), k, v, c.table, c.seq_lens, c.k, c.ks, c.v, c.vs, starts(new), ws=ws)
        assert dsa.read_error(ws) == 0
        return k, v

    g = torch.Generator().manual_seed(d)
    small = lambda: 0.02 * torch.randn((2, d), generator=g)  # noqa: E731
    zero, one = torch.zeros((2, d)), torch.zeros((2, d))
    one[1, 5] = 448.0  # head 1: a value whose scale is 1
    first = lambda x: int(c.table[x, 0])  # noqa: E731
    for _ in range(9):  # sequence 0: zeros; 1: head 1 has a value; 2: the keys alone are zeros
        append(([zero, one, -zero], [-zero, zero, one + 1.0]), [1, 1, 1])
    assert bool((c.ks[[first(0), first(1), first(2)]] == 1.0).all())
    k, v = append(([small() for _ in range(3)], [small() for _ in range(3)]), [1, 1, 1])
    top = lambda x: (x.cpu().float().abs().amax(-1) / 448.0).cuda()  # noqa: E731  (a quotient: on the GPU torch multiplies by 1 / 448)
    assert torch.equal(c.ks[first(0)], top(k[0])) and torch.equal(c.vs[first(0)], top(v[0]))
    assert torch.equal(c.ks[first(1), :1], top(k[1, :1])) and float(c.ks[first(1), 1]) == 1.0 and torch.equal(c.vs[first(1)], top(v[1]))
    assert torch.equal(c.ks[first(2)], top(k[2])) and torch.equal(c.vs[first(2)], top((one + 1.0).to(ACT[type])))
    for x, codes, scale in ((k, c.k, c.ks), (v, c.v, c.vs)):
        for b in range(3):
            s = scale[first(b)]
            want = (x[b].float().cpu() / s.cpu()[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            assert torch.equal(codes[first(b), :, 9].cpu(), want)
    assert not (c.k[first(0), :, :9] & 0x7F).any() and not (c.v[first(0), :, :9] & 0x7F).any()
    append_and_check(c, [120, 3, 70])  # and on as ever
    q = c.queries(3)
    check(c, q, [1, 1, 1], attend(c, q, [1, 1, 1], 0.1), 0.1)


def test_append_of_the_smallest_values():
    """Magnitudes whose 448th part is 0 in fp32: a scale of 1 and codes of 0, not a scale of 0 and NaN."""
    for spread in (1e-44, 1e-42, 3e-39):
        c = Cache([0, 0, 70], 2, 1, 16, 32, "f32", seed=27, room=[140, 140, 140])
        append_and_check(c, [65, 3, 60], spread=spread)
        append_and_check(c, [1, 1, 1], spread=spread)
        assert bool((c.ks[c.table[:, 0].long()] > 0).all()) and not (value(c.k[c.table[1, 0].long(), 0, :4])).isnan().any()


def test_append_faults():
    c = Cache([10, 20, 30], 4, 2, 32, 32, "bf16", seed=25, room=[80, 80, 80])
    k, v = (torch.randn((3, 2, 32), device="cuda").bfloat16() for _ in range(2))
    ws = dsa.grouped_workspace(c.dims(), 8)
    call = lambda lens, cu=None, table=c.table, k=k, v=v: dsa.grouped_append(c.dims(), k, v, table, ints(lens), c.k, c.ks, c.v, c.vs,  # noqa: E731
                                                                             None if cu is None else ints(cu), ws=ws)
    before = [t.clone() for t in (c.k, c.ks, c.v, c.vs)]
    untouched = lambda: all(same(a, b) for a, b in zip((c.k, c.ks, c.v, c.vs), before))  # noqa: E731
    call([0, 0, 0], [0, 0, 0, 0], k=k[:0], v=v[:0])
    assert dsa.read_error(ws) == 0 and untouched()
    call([11, 21, 31], [0, 0, 4, 3])
    assert dsa.read_error(ws) == 2 and untouched()
    call([-1, c.width * 64 + 1, 1 << 30])
    assert dsa.read_error(ws) == 2 and untouched()
    bad = c.table.clone()
    bad[0, 0], bad[1, 0], bad[2, 0] = -1, c.blocks, -(1 << 31)
    call([11, 21, 31], table=bad)
    assert dsa.read_error(ws) == 1 and untouched()
    # more new tokens than positions: the first are skipped
    call([11, 21, 2], [0, 0, 0, 3])
    assert dsa.read_error(ws) == 2
    blk = int(c.table[2, 0])
    for got, x, scale in ((c.k, k, c.ks), (c.v, v, c.vs)):
        y = value(got[blk, :, :2]) * scale[blk].double()[:, None, None]
        assert bool(((y - x[1:].double().transpose(0, 1)).abs() <= 0.07 * x.double().abs().amax()).all())
    keep = torch.ones(c.blocks, dtype=torch.bool, device="cuda")
    keep[blk] = False
    assert all(same(a[keep], b[keep]) for a, b in zip((c.k, c.ks, c.v, c.vs), before))


# ------------------------------------------------------------------------------------------------ eviction

def expected_kept(w, n, keep, sink, recent):
    """Ascending positions of one sequence and head (a list)."""
    if n <= keep:
        return list(range(n))
    w = [(-math.inf if x != x else x) for x in w[:n].tolist()]
    rest = sorted(range(sink, n - recent), key=lambda i: (-w[i], i))[:keep - sink - recent]
    return sorted(list(range(sink)) + list(range(n - recent, n)) + rest)


def evict_and_check(c, w, keep, sink, recent, faults=0, new_table=None, extra=0):
    B, blocks = len(c.lens), (keep + 63) // 64 + extra
    if new_table is None:  # new blocks behind the old ones
        more = B * blocks
        new_table = (c.blocks + torch.randperm(more, generator=c.g, device="cuda")).to(torch.int32).view(B, blocks)
        for name, fill in (("k", NAN_CODE), ("v", NAN_CODE), ("ks", float("nan")), ("vs", float("nan"))):
            t = getattr(c, name)
            setattr(c, name, torch.cat([t, torch.full((more,) + t.shape[1:], fill, dtype=t.dtype, device="cuda")]))
        c.blocks += more
    want = [t.cpu().clone() for t in (c.k, c.ks, c.v, c.vs)]
    table, to, w_cpu = c.table.cpu(), new_table.cpu(), w.cpu()
    ws = dsa.grouped_workspace(c.dims(), B)
    kept, lens, w_out = dsa.grouped_evict(c.dims(), w, keep, c.table, c.seq_lens, new_table, c.k, c.ks, c.v, c.vs, sink=sink, recent=recent, ws=ws)
    assert dsa.read_error(ws) == faults
    assert lens.tolist() == [min(n, keep) for n in c.lens]
    kept, w_out = kept.cpu(), w_out.cpu()
    for b, n in enumerate(c.lens):
        m = min(n, keep)
        for h in range(c.H_kv):
            at = expected_kept(w_cpu[b, h], n, keep, sink, recent)
            assert kept[b, h].tolist() == at + [-1] * (keep - m)
            assert same(w_out[b, h, :m], w_cpu[b, h, at]) and not w_out[b, h, m:].any()
            for codes, scale in ((want[0], want[1]), (want[2], want[3])):
                for j in range(0, m, 64):
                    i = torch.tensor(at[j:j + 64])
                    old, dst = table[b].long()[i // 64], int(to[b, j // 64])
                    ok = (old >= 0) & (old < c.blocks)
                    if not 0 <= dst < c.blocks:
                        continue
                    src = codes[old.clamp(0, c.blocks - 1), h, i % 64]
                    s = scale[old.clamp(0, c.blocks - 1), h]
                    if n > keep:
                        x = src.view(torch.float8_e4m3fn).float() * s[:, None]
                        top = x[ok].abs().max() / 448.0 if ok.any() else torch.tensor(0.0)
                        new = top if top > 0 else torch.tensor(1.0)
                        src = (x / new).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                        scale[dst, h] = new
                    elif ok[0]:
                        scale[dst, h] = s[0]
                    codes[dst, h, :len(i)][ok] = src[ok]
    for got, ref in zip((c.k, c.ks, c.v, c.vs), want):
        assert same(got, ref)
    c.table, c.width, c.lens, c.seq_lens = new_table, new_table.shape[1], lens.tolist(), lens
    return kept, w_out.cuda()


@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (64, 4, 10), (100, 0, 100), (129, 129, 0), (300, 1, 37), (300, 150, 150), (700, 3, 0)])
def test_evict(keep, sink, recent):
    for H_kv, d_qk, d_v in ((2, 128, 128), (3, 16, 80), (1, 256, 192)):
        c = Cache([700, 1, 0, 300, 301, 64, 1500], 6, H_kv, d_qk, d_v, seed=keep + d_qk)
        w = torch.randn((7, H_kv, c.width * 64), generator=c.g, device="cuda").mul_(2).exp_()
        evict_and_check(c, w, keep, sink, recent, extra=keep % 2)


def test_evict_ties_and_special_weights():
    c = Cache([500] * 6, 2, 1, 16, 16, seed=31)
    w = torch.zeros((6, 1, c.width * 64), device="cuda")
    w[1] = torch.arange(w.shape[2], device="cuda") % 3
    w[2] = -1.0
    w[2, 0, ::5] = -0.0
    w[2, 0, 1::5] = 0.0
    w[3] = float("nan")
    w[3, 0, ::7] = -math.inf
    w[3, 0, 3::50] = math.inf
    w[4] = torch.rand_like(w[4]) * 1e-42  # subnormal
    w[5] = 1.0 + torch.randint(0, 4, w[5].shape, device="cuda") * 2.0 ** -23
    for keep in (100, 250, 499):
        evict_and_check(Cache([500] * 6, 2, 1, 16, 16, seed=31), w, keep, 5, 20)


def test_evict_of_the_smallest_values():
    """Kept rows whose largest magnitude has 0 for its 448th part."""
    c = Cache([300, 200], 2, 1, 16, 32, seed=36)
    for t, scale in ((c.k, c.ks), (c.v, c.vs)):
        used = torch.cat([c.table[0, :5], c.table[1, :4]]).long()
        t[used] &= 0xBF  # codes below 2
        scale[used] = 2.0 ** -149
    w = torch.rand((2, 1, c.width * 64), generator=c.g, device="cuda")
    to = torch.arange(c.blocks, c.blocks + 4, dtype=torch.int32, device="cuda").view(2, 2)
    for name, fill in (("k", NAN_CODE), ("v", NAN_CODE), ("ks", float("nan")), ("vs", float("nan"))):
        t = getattr(c, name)
        setattr(c, name, torch.cat([t, torch.full((4,) + t.shape[1:], fill, dtype=t.dtype, device="cuda")]))
    c.blocks += 4
    evict_and_check(c, w, 100, 2, 8, new_table=to)
    assert bool((c.ks[to.long()] == 1.0).all()) and not value(c.k[to[:, 0].long()]).isnan().any()


def test_evict_long_sequences():
    c = Cache([70000, 20000], 2, 1, 16, 16, seed=32)
    w = torch.randn((2, 1, c.width * 64), generator=c.g, device="cuda").exp_()
    evict_and_check(c, w, 33000, 16, 500)


def test_evict_in_place_and_faults():
    """A sequence that is not cut may keep its blocks; rows from and into invalid blocks are skipped."""
    c = Cache([100, 400, 64], 4, 2, 32, 32, seed=33, room=[100, 900, 64])
    w = torch.rand((3, 2, c.width * 64), generator=c.g, device="cuda")
    to = c.table[:, :4].clone()
    to[1] = c.table[1, 7:11]
    evict_and_check(c, w, 200, 2, 8, new_table=to)
    c = Cache([100, 400, 300], 4, 2, 32, 32, seed=34, room=[100, 900, 900])
    w = torch.rand((3, 2, c.width * 64), generator=c.g, device="cuda")
    c.table[1, 2], c.table[0, 1] = -1, c.blocks
    to = c.table[:, 7:11].clone()
    to[0], to[2, 1] = c.free[:1].expand(4), 1 << 20
    to[0, 0] = c.free[1]
    evict_and_check(c, w, 200, 2, 8, new_table=to, faults=1)
    c = Cache([100, 400, 64], 4, 2, 32, 32, seed=35, room=[100, 900, 64])
    c.seq_lens = ints([100, -5, c.width * 64 + 1])
    c.lens = [100, 0, 0]
    evict_and_check(c, torch.rand((3, 2, c.width * 64), device="cuda"), 200, 2, 8, faults=2)


def test_rows_of_another_width_are_refused():
    """Tables, weights and kept positions of more dimensions whose rows are longer than the call reads them."""
    c = Cache([100, 70], 4, 2, 32, 32, seed=37, room=[200, 200])
    gd, ws = c.dims(), dsa.grouped_workspace(c.dims(), 2, weights=True)
    q, kv = c.queries(2), torch.randn((2, 2, 32), device="cuda").bfloat16()
    w = torch.zeros((2, 2, c.width * 64), device="cuda")
    wide = lambda t: torch.cat([t, t[..., :64]], -1).contiguous()  # noqa: E731
    to, before = c.table[:, 2:4].contiguous(), [t.clone() for t in (c.k, c.ks, c.v, c.vs)]
    append = lambda t=c.table: dsa.grouped_append(gd, kv, kv, t, c.seq_lens, c.k, c.ks, c.v, c.vs, ws=ws)  # noqa: E731
    attn = lambda t=c.table, **kw: dsa.grouped_attn(gd, q, c.k, c.ks, c.v, c.vs, t, c.seq_lens, 0.1, ws=ws, **kw)  # noqa: E731
    evict = lambda t=c.table, w=w, **kw: dsa.grouped_evict(gd, w, 64, t, c.seq_lens, to, c.k, c.ks, c.v, c.vs, ws=ws, **kw)  # noqa: E731
    for call, what in ((lambda: append(wide(c.table)), "block_table"), (lambda: attn(wide(c.table)), "block_table"),
                       (lambda: evict(wide(c.table)), "block_table"), (lambda: attn(weights=wide(w)), "weights"),
                       (lambda: attn(weights_out=wide(w)), "weights_out"), (lambda: evict(w=wide(w)), "weights"),
                       (lambda: evict(weights_out=torch.empty((2, 2, 192), device="cuda")), "weights_out"),
                       (lambda: evict(kept=torch.empty((2, 2, 65), dtype=torch.int32, device="cuda")), "kept")):
        with pytest.raises(ValueError, match="rows of " + what):
            call()
    assert all(same(a, b) for a, b in zip((c.k, c.ks, c.v, c.vs), before))
    ref = attn(weights=w.clone())
    got = attn(c.table.flatten(), weights=w.flatten())  # without dimensions of their own
    assert torch.equal(got[0], ref[0]) and dsa.read_error(ws) == 0
    # the same rows in other dimensions, and more of them
    for weights in (w.view(2, 2, -1, 64), w.view(2, -1), w.view(4, -1), torch.cat([w, w]), torch.cat([w, w]).view(4, 2, -1, 64)):
        for table in (c.table, torch.cat([c.table, c.table])):
            got = attn(table, weights=weights.clone())
            assert torch.equal(got[0], ref[0]) and dsa.read_error(ws) == 0


# ------------------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_decode_loop_with_eviction(type):
    """A prompt appended, decode steps that append, attend and count weights, an eviction, and further steps on what is left,
    with drafts that are dropped again by a shorter length."""
    H, H_kv, d = 8, 2, 64
    lens = [150, 70, 0]
    c = Cache([0, 0, 0], H, H_kv, d, d, type, seed=41, room=[400, 400, 400])
    append_and_check(c, lens)
    w = torch.zeros((3, H_kv, c.width * 64), device="cuda")

    def step(new):
        nonlocal w
        append_and_check(c, new)
        q = c.queries(sum(new), 2.0)
        before = w.clone()
        check(c, q, new, attend(c, q, new, d ** -0.5, weights=w), d ** -0.5, before, w)

    for i in range(5):
        step([1, 1, 1])
    step([4, 2, 3])
    c.lens = [n - m for n, m in zip(c.lens, [2, 0, 3])]  # rejected drafts
    c.seq_lens = ints(c.lens)
    step([1, 1, 1])
    blocks = 3
    new_table = c.table[:, -1 - blocks:-1].clone()
    _, w = evict_and_check(c, w, 80, 4, 16, new_table=new_table)
    assert max(c.lens) == 80
    for i in range(3):
        step([1, 1, 1])
    step([5, 1, 2])


# ------------------------------------------------------------------------------------------------ value scales that lie apart

def light_and_heavy(type, H, n, d_v=32, new=1, seed=50):
    """One sequence of n positions whose logits are 0 but for those set by `louder`: head h of H multiplies that by its own gap."""
    c = Cache([n], H, 1, 16, d_v, type, seed=seed)
    at = c.table[0, :(n + 63) // 64].long()
    c.k[at] = 0
    c.ks[at] = 1.0
    c.v[at] &= 0x7F  # all of one sign: errors of one sign would add up
    q = torch.zeros((new, H, 16), dtype=ACT[type], device="cuda")
    q[..., 0] = (torch.linspace(0.0, 20.0, H, device="cuda") * math.log(2.0)).to(ACT[type])
    return c, q, at


def louder(c, pos):
    c.k[int(c.table[0, pos // 64]), 0, pos % 64, 0] = 0x38  # 1.0


SHAPES = [("f32", 8, 1), ("f32", 16, 1), ("bf16", 8, 1), ("bf16", 16, 1), ("bf16", 32, 1), ("bf16", 64, 1), ("bf16", 8, 7)]


@pytest.mark.parametrize("type,H,new", SHAPES)
@pytest.mark.parametrize("value,block", [(0.1, 0), (0.02, 1), (0.005, 37), (0.02, 68)])
def test_a_heavy_block_of_zeros_beside_small_values(type, H, new, value, block):
    """A block of zero values, whose scale is 1, takes up to all but a millionth of a row's weight; the others' small values
    are held against their own scales."""
    n = 69 * 64 - 5
    c, q, at = light_and_heavy(type, H, n, new=new)
    c.vs[at] = value / 448
    c.v[at[block]] = 0
    c.vs[at[block]] = 1.0
    for pos in range(64 * block, min(64 * block + 64, n)):
        louder(c, pos)
    w = torch.zeros((1, 1, c.width * 64), device="cuda")
    got = attend(c, q, [new], 1.0, weights_out=w)
    check(c, q, [new], got, 1.0, None, w)


@pytest.mark.parametrize("type,H,new", SHAPES)
def test_a_heavy_position_in_a_block_of_large_values(type, H, new):
    """A position of zero values that takes most of the weight, in a block that a single value of another one gives a large
    scale: the columns without that value keep the light positions' weights."""
    for block in (0, 1, 30):
        c, q, at = light_and_heavy(type, H, 64 * 64, new=new)
        c.vs[at] = 2.0 ** -13
        c.v[at[block]] = 0
        c.v[at[block], 0, 9, 0] = 0x7E  # 448
        c.vs[at[block]] = 1.0
        louder(c, 64 * block + 3)
        check(c, q, [new], attend(c, q, [new], 1.0), 1.0)


@pytest.mark.parametrize("type,H,new", SHAPES)
def test_scales_that_change_from_block_to_block(type, H, new):
    """Blocks with scales far apart in turn (also with the smaller ones first, and with invalid blocks between them); large
    values stand in one column, so that the others have the small ones alone."""
    for first, gone in ((0, ()), (1, ()), (0, (6, 9, 20))):
        c, q, at = light_and_heavy(type, H, 50 * 64 - 30, new=new)
        c.vs[at] = 2.0 ** -13
        large = at[first::2]
        c.v[large, :, :, 1:] = 0
        c.vs[large] = 3.0
        for pos in (70, 200, 2000):
            louder(c, pos)
        for j in gone:
            c.table[0, j] = -1
        w = torch.rand((1, 1, c.width * 64), device="cuda")
        base = w.clone()
        got = attend(c, q, [new], 1.0, faults=1 if gone else 0, weights=w)
        check(c, q, [new], got, 1.0, base, w)


@pytest.mark.parametrize("type,H,new", SHAPES)
def test_scales_of_any_size(type, H, new):
    """Value scales near both ends of their range, alone, and 2^50 and more apart: the largest ones' columns are right, and the
    smaller ones' too as far as 2^60 below."""
    for low, high in ((-88, -88), (100, 100), (60, 110), (-88, -40), (-20, 70)):
        c, q, at = light_and_heavy(type, H, 30 * 64 - 7, new=new)
        c.vs[at] = 2.0 ** high
        c.vs[at[::3]] = 2.0 ** low
        if low != high:  # the small blocks alone have columns of their own
            other = torch.ones(30, dtype=torch.bool, device="cuda")
            other[::3] = False
            c.v[at[other], :, :, :8] = 0
        louder(c, 100)
        out, lse = attend(c, q, [new], 1.0)
        cols = range(8, 32) if high - low > 60 else range(32)
        for scale, part in ((high, [e for e in cols if e >= 8]), (low, [e for e in cols if e < 8])):
            k, v, ok = c.rows(0, 0)
            for i in range(new):
                p = torch.softmax((q[i].double() @ k.T).masked_fill(torch.arange(len(k), device="cuda") > len(k) - new + i, -math.inf), -1)
                want = (p @ v)[:, part] * 2.0 ** -scale
                # as for scales that rise and fall
                rel = (2.0 ** -10 + 2.0 ** -8 if type == "bf16" else 2.0 ** -21) + 2 * 2.0 ** -22 * 15 + len(k) * 2.0 ** -24
                tol = rel * want + (2.0 ** -22 if type == "bf16" else 2.0 ** -30) * p.amax(-1, keepdim=True) * v.sum(0)[part] * 2.0 ** -scale
                assert bool(((out[i][:, part].double() * 2.0 ** -scale - want).abs() <= tol).all()), (low, high, scale)


@pytest.mark.parametrize("type,H,new", SHAPES)
@pytest.mark.parametrize("step", [1.25, -1.25, 0.5, -2.5])
def test_scales_that_rise_and_fall_by_steps(type, H, new, step):
    """Scales that drift by a few powers of two a block, up or down, up to 2^54 in all; block j has values in column j % 32 alone."""
    blocks = 44 if abs(step) < 2 else 22
    c, q, at = light_and_heavy(type, H, 64 * blocks, new=new)
    for j in range(blocks):
        keep = c.v[at[j], :, :, j % 32].clone()
        c.v[at[j]] = 0
        c.v[at[j], :, :, j % 32] = keep
        c.vs[at[j]] = 2.0 ** (step * (j - blocks // 2)) / 448
    for pos in (3, 64 * blocks - 9 - new):
        louder(c, pos)
    out, _ = attend(c, q, [new], 1.0)
    k, v, _ = c.rows(0, 0)
    for i in range(new):
        z = (q[i].double() @ k.T).masked_fill(torch.arange(64 * blocks, device="cuda") > 64 * blocks - new + i, -math.inf)
        p = torch.softmax(z, -1)
        # the header's bounds: 11 bits of a weight in bf16 and 2^-22 of the row's largest, in fp32 24 bits and 2^-30; logits of one
        # product each, up to 14 (20 ln 2): 2^-22 of that in the factor and the subtraction, twice (logit and sum); the sums' roundings
        rel = (2.0 ** -10 + 2.0 ** -8 if type == "bf16" else 2.0 ** -21) + 2 * 2.0 ** -22 * 15 + 64 * blocks * 2.0 ** -24
        tol = rel * (p @ v) + (2.0 ** -22 if type == "bf16" else 2.0 ** -30) * p.amax(-1, keepdim=True) * v.sum(0) + 1e-30
        err = (out[i].double() - p @ v).abs()
        assert bool((err <= tol).all()), (i, float((err / tol).max()))


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_rotation_goes_on_over_an_eviction(type):
    """Tokens rotated at their own positions before and after an eviction: the logit of a query at p with a key of s is the
    cosine of p - s, although the cache counts fewer positions."""
    H, H_kv, d, keep, sm = 4, 2, 64, 80, 2.0
    lens = [150, 90]
    c = Cache([0, 0], H, H_kv, d, d, type, seed=51, room=[400, 400])
    freq = torch.zeros(d // 2, dtype=torch.float64, device="cuda")
    freq[0] = 1.0
    gd, ws = c.dims(), dsa.grouped_workspace(c.dims(), 300, weights=True)

    def rows(pos, heads):  # 1 in the first column, turned by the position
        x = torch.zeros((len(pos), heads, d), dtype=ACT[type], device="cuda")
        x[..., 0] = 1.0
        return dsa.rope(x, freq, q_pos=ints(pos), layout="half")

    pos = list(range(150)) + list(range(90))
    table, at = c.table, [torch.arange(n, device="cuda").expand(H_kv, n) for n in lens]  # own positions of the cached rows
    seq_lens = ints(lens)
    dsa.grouped_append(gd, rows(pos, H_kv), rows(pos, H_kv), table, seq_lens, c.k, c.ks, c.v, c.vs, starts(lens), ws=ws)
    w = torch.rand((2, H_kv, c.width * 64), device="cuda")
    new_table = c.table[:, -4:-2].contiguous()
    kept, seq_lens, w = dsa.grouped_evict(gd, w, keep, table, seq_lens, new_table, c.k, c.ks, c.v, c.vs, sink=2, recent=8, ws=ws)
    assert seq_lens.tolist() == [keep, keep]
    at = [kept[b].long() for b in range(2)]
    gd = dsa.grouped_dims(type, 2, new_table.shape[1], c.blocks, H, H_kv, d, d)
    for step in range(3):
        own = [n + step for n in lens]
        seq_lens += 1
        at = [torch.cat([a, torch.full((H_kv, 1), p, device="cuda")], 1) for a, p in zip(at, own)]
        x = rows(own, H_kv)
        dsa.grouped_append(gd, x, x, new_table, seq_lens, c.k, c.ks, c.v, c.vs, ws=ws)
        got = torch.zeros_like(w)
        dsa.grouped_attn(gd, rows(own, H), c.k, c.ks, c.v, c.vs, new_table, seq_lens, sm, weights_out=got, ws=ws)
        assert dsa.read_error(ws) == 0
        for b in range(2):
            want = torch.softmax(sm * torch.cos((own[b] - at[b]).double()), -1) * (H // H_kv)
            # a cached element was rounded three times at most, each by 2^-4 of it (or a step of the smallest codes, 2^-10 of a scale
            # of 1 / 448), after bf16's 2^-8: a logit is off by 2 * 0.2, and the sum with it
            off = (got[b, :, :want.shape[1]].double() / want).log().abs().max()
            assert float(off) <= 2 * sm * 0.2, (step, b, float(off))


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_two_graphs_share_a_workspace(type):
    """A decode step (append, attention, weights) and an eviction, captured apart with one workspace, replayed in turn on new
    inputs: what the same calls give one by one."""
    H, H_kv, d, keep = 8, 2, 64, 300
    c = Cache([900, 40, 2000], H, H_kv, d, d, type, seed=52, room=[1000, 1000, 2100])
    c.vs *= torch.exp2(4.0 * torch.randn(c.vs.shape, generator=c.g, device="cuda"))
    gd, ws = c.dims(), dsa.grouped_workspace(c.dims(), 3, weights=True)
    to = (c.blocks + torch.arange(15, device="cuda")).to(torch.int32).view(3, 5)
    for name in ("k", "v", "ks", "vs"):
        t = getattr(c, name)
        setattr(c, name, torch.cat([t, t[:15]]))
    gd.num_blocks += 15
    x = [c.queries(3)[:, :H_kv].contiguous() for _ in range(2)]
    q, w = c.queries(3), torch.rand((3, H_kv, c.width * 64), device="cuda")
    kept, lens, left = torch.empty((3, H_kv, keep), dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty((3, H_kv, 320), device="cuda")
    out, lse = torch.empty((3, H, d), dtype=ACT[type], device="cuda"), torch.empty((3, H), device="cuda")

    def step():
        dsa.grouped_append(gd, *x, c.table, c.seq_lens, c.k, c.ks, c.v, c.vs, ws=ws)
        dsa.grouped_attn(gd, q, *c.args(), 0.125, weights=w, out=out, lse=lse, ws=ws)

    def evict():
        dsa.grouped_evict(gd, w, keep, c.table, c.seq_lens, to, c.k, c.ks, c.v, c.vs, sink=4, recent=30, kept=kept, new_lens=lens, weights_out=left, ws=ws)

    state = [c.k, c.ks, c.v, c.vs, w, out, lse, kept, lens, left]
    graphs, side = [torch.cuda.CUDAGraph() for _ in range(2)], torch.cuda.Stream()
    step(), evict()  # (what a first call sets up)
    torch.cuda.synchronize()
    for g, call in zip(graphs, (step, evict)):
        with torch.cuda.graph(g, stream=side):
            call()
    torch.cuda.synchronize()
    start = [t.clone() for t in state]
    for turn in range(3):
        q.copy_(c.queries(3))
        for t in x:
            t.copy_(c.queries(3)[:, :H_kv])
        c.seq_lens += 1
        for t, s in zip(state, start):
            t.copy_(s)
        step(), evict()
        want = [t.clone() for t in state]
        for t, s in zip(state, start):
            t.copy_(s)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert all(same(t, s) for t, s in zip(state, want)), turn
        start = want
    assert dsa.read_error(ws) == 0 and not ws[:256].any()
