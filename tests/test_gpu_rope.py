"""dsa_rope and dsa_cache_append_rope against the rotation in 64 bits: both layouts, parts of heads, far
positions, strided views, in place and out of place, the transpose, and the append's rounding per mode."""
import math

import numpy as np
import pytest
import torch

import indexer_top_sparse_paged_gb300 as dsa
import workloads as W
from cases import small_spec

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
# cos and sin of the fp32 fraction: half an ulp of a fraction below 1/2 turn (2 pi 2^-26) and two ulp of the
# function, then three roundings of products and sum: below 5e-7 of |u| + |v|
ARITH = 5e-7


def rotated64(x, pos, freq, layout, scale=1.0, transpose=False):
    """(y, |u| + |v| per element) in fp64; rows with a negative position unchanged."""
    x = x.double()
    ang = pos.double()[:, None] * freq
    c, s = (scale * ang.cos())[:, None], (scale * ang.sin())[:, None]
    if transpose:
        s = -s
    h = x.shape[-1] // 2
    u, v = (x[..., :h], x[..., h:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])
    a, b, m = u * c - v * s, u * s + v * c, u.abs() + v.abs()
    join = (lambda p, q: torch.cat((p, q), -1)) if layout == "half" else (lambda p, q: torch.stack((p, q), -1).flatten(-2))
    keep = (pos < 0)[:, None, None]
    return torch.where(keep, x, join(a, b)), torch.where(keep, 0.0, join(m, m))


def check(y, x, pos, freq, layout, scale=1.0, transpose=False):
    want, mag = rotated64(x, pos, freq, layout, scale, transpose)
    tol = want.abs() * HALF_STEP[y.dtype] + abs(scale) * ARITH * mag * (1 + HALF_STEP[y.dtype])
    # a value at the edge of two binades rounds by the upper one's half step
    assert bool(((y.double() - want).abs() <= tol * (1 + 2.0 ** -7)).all()), float(((y.double() - want).abs() - tol).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,H,rot", [(1, 1, 2), (1, 128, 64), (3, 7, 6), (33, 8, 96), (257, 64, 64), (5, 3, 512), (40, 1, 128), (9, 5, 48)])
def test_rope_in_place_and_out_of_place(dtype, layout, T, H, rot):
    g = torch.Generator(device="cuda").manual_seed(T * 131 + H + rot)
    x = torch.randn((T, H, rot), generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda").to(torch.int32)
    pos[0] = 0 if T > 1 else (1 << 31) - 1
    freq = dsa.rope_frequencies(rot, scaling="yarn", factor=40.0)
    keep = x.clone()
    out = torch.empty_like(x)
    assert dsa.rope(x, freq, q_pos=pos, layout=layout, out=out, scale=1.25) is out
    assert torch.equal(x, keep)
    check(out, x, pos, freq, layout, 1.25)
    assert dsa.rope(x, freq, q_pos=pos, layout=layout, scale=1.25) is x
    assert torch.equal(x, out)
    assert dsa.last_launch_count() == 1


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("off", [0, 1, 3, 8, 64])
def test_rope_part_of_wider_heads(dtype, off):
    """Views at any offset, in and out of unlike strides; the columns around them are left as they were."""
    T, H, rot = 37, 6, 64
    x = torch.randn((T, H, 130), device="cuda").to(dtype)
    q = torch.randn((H, T, 129), device="cuda").to(dtype).transpose(0, 1)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 977
    freq = dsa.rope_frequencies(rot)
    keep_q, keep_x = q.clone(), x.clone()
    for layout in ("interleaved", "half"):
        dsa.rope(x[..., off:off + rot], freq, q_pos=pos, layout=layout, out=q[..., off:off + rot])
        check(q[..., off:off + rot], x[..., off:off + rot], pos, freq, layout)
        assert torch.equal(q[..., :off], keep_q[..., :off]) and torch.equal(q[..., off + rot:], keep_q[..., off + rot:])
        assert torch.equal(x, keep_x)
        dsa.rope(x[:, 1:4, off:off + rot], freq, q_pos=pos, layout=layout)
        check(x[:, 1:4, off:off + rot], keep_x[:, 1:4, off:off + rot], pos, freq, layout)
        x[:, 1:4, off:off + rot] = keep_x[:, 1:4, off:off + rot]
        assert torch.equal(x, keep_x)


def test_rope_several_tensors_decode_positions_and_empty_sequences():
    B, rot = 9, 64
    lens = torch.tensor([1, 0, 5, 1 << 20, 64, 0, 7, 2, 30000], dtype=torch.int32, device="cuda")
    q, qi = torch.randn((B, 128, rot), device="cuda").bfloat16(), torch.randn((B, 64, rot), device="cuda").bfloat16()
    none = torch.empty((B, 0, rot), device="cuda").bfloat16()
    freq = dsa.rope_frequencies(rot)
    a, b, c = q.clone(), qi.clone(), none
    got = dsa.rope([a, c, b], freq, lens, layout=["interleaved", "half", "half"])
    assert got[0] is a and got[2] is b and dsa.last_launch_count() == 1
    check(a, q, lens - 1, freq, "interleaved")
    check(b, qi, lens - 1, freq, "half")
    empty = (lens == 0)
    assert torch.equal(a[empty], q[empty]) and torch.equal(b[empty], qi[empty])
    dsa.rope(q[:0], freq, q_pos=lens[:0])  # no rows: nothing is launched
    assert dsa.last_launch_count() == 0


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_gradient_is_the_transpose(layout):
    """<dy, J dx> by differences of the forward call and <J^T dy, dx> by the transposed one: the rotation is
    linear, so both are equal up to fp32 roundings of n products of order 1."""
    T, H, rot, n = 11, 3, 32, 11 * 3 * 32
    freq = dsa.rope_frequencies(rot)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 5021
    x, dx, dy = (torch.randn((T, H, rot), device="cuda") for _ in range(3))
    f = lambda v: dsa.rope(v.clone(), freq, q_pos=pos, layout=layout, scale=0.7).double()  # noqa: E731
    num = ((f(x + dx) - f(x - dx)) / 2 * dy.double()).sum()
    back = dsa.rope(dy.clone(), freq, q_pos=pos, layout=layout, scale=0.7, transpose=True)
    check(back, dy, pos, freq, layout, 0.7, True)
    assert abs(float(num - (back.double() * dx.double()).sum())) <= n * 64 * 2.0 ** -24
    both = dsa.rope(dsa.rope(x.clone(), freq, q_pos=pos, layout=layout), freq, q_pos=pos, layout=layout, transpose=True)
    assert float((both - x).abs().max()) <= 4 * ARITH * float(x.abs().max()) * 2


def test_rope_frequencies_of_every_scaling():
    rot, base, factor, L = 64, 10000.0, 40.0, 4096.0
    i = np.arange(rot // 2, dtype=np.float64)
    plain = base ** (-2 * i / rot)
    np.testing.assert_allclose(dsa.rope_frequencies(rot, base).cpu().numpy(), plain, rtol=1e-14)
    np.testing.assert_allclose(dsa.rope_frequencies(rot, base, factor=8.0).cpu().numpy(), plain / 8, rtol=1e-14)
    b = dsa.rope_frequencies(rot, base, scaling="base", factor=factor).cpu().numpy()
    np.testing.assert_allclose(b, (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot), rtol=1e-14)
    assert b[0] == 1.0 and abs(b[-1] * factor / plain[-1] - 1) < 1e-12
    y = dsa.rope_frequencies(rot, base, scaling="yarn", factor=factor, original_length=L).cpu().numpy()
    turns = L * plain / (2 * math.pi)
    assert np.allclose(y[turns > 34], plain[turns > 34], rtol=1e-14)           # above beta_fast: kept
    assert np.allclose(y[turns < 0.7], plain[turns < 0.7] / factor, rtol=1e-14)  # below beta_slow: stretched
    assert np.all(np.diff(y) < 0) and np.all(y <= plain * (1 + 1e-15)) and np.all(y >= plain / factor * (1 - 1e-14))


def test_rope_on_another_stream_and_in_a_graph():
    T, rot = 64, 64
    freq = dsa.rope_frequencies(rot)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    x = torch.randn((T, 16, rot), device="cuda").bfloat16()
    out = torch.zeros_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dsa.rope(x, freq, q_pos=pos, out=out, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    check(out, x, pos, freq, "interleaved")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.rope(x, freq, q_pos=pos, out=out)
    x.normal_()
    pos.add_(100)
    out.zero_()
    g.replay()
    check(out, x, pos, freq, "interleaved")


# ------------------------------------------------------------------------------------ rotated append

def _dev(a):
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).cuda().view(torch.bfloat16)
    return torch.from_numpy(a).cuda()


class Append:
    def __init__(self, mode, kv, lens, new, seed, **kw):
        spec = small_spec(mode, lens, 64, new_tokens=new, kv=kv, **kw)
        c = self.case = W.generate(spec, seed=seed)
        s = c.spec
        self.dims = dsa.make_dims(s.mode, s.B, c.max_blocks, c.num_blocks, s.H_I, s.d_I, s.H, s.d, s.d_v, s.K, kv=s.kv)
        act = torch.float32 if mode == "f32" else torch.bfloat16
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.k_new = (3 * torch.randn((s.T, s.d_I), generator=g, device="cuda")).to(act)
        self.kv_new = torch.randn((s.T, s.d), generator=g, device="cuda").to(act)
        self.table, self.lens = _dev(c.block_table), _dev(c.seq_lens)
        self.q_seq, self.q_pos = _dev(c.q_seq), _dev(c.q_pos)
        self.ws = dsa.workspace(self.dims, 1)

    def caches(self):
        c = self.case
        return _dev(c.k_I), None if c.k_I_scale is None else _dev(c.k_I_scale), _dev(c.kv)

    def rows(self):
        s, p = self.q_seq.long(), self.q_pos.long()
        return self.table[s, p // 64].long() * 64 + p % 64


SHAPES = {"f32": dict(H_I=8, d_I=36, H=4, d=68, d_v=48), "bf16": {}, "bf16_kfp8": {}, "mxfp8": {}}
MODES = [("f32", "act"), ("bf16", "act"), ("bf16", "fp8"), ("bf16_kfp8", "act"), ("bf16_kfp8", "fp8"), ("mxfp8", "fp8")]


@pytest.mark.parametrize("mode,kv", MODES)
@pytest.mark.parametrize("decode", [True, False])
def test_append_without_rotation_is_the_plain_append(mode, kv, decode):
    lens, new = ([1, 63, 64, 65, 128, 500], None) if decode else ([300, 1000, 77, 400], [150, 1, 13, 200])
    p = Append(mode, kv, lens, new, 400, **SHAPES[mode])
    a, b = p.caches(), p.caches()
    freq = dsa.rope_frequencies(16)
    rows = (None, None) if decode else (p.q_seq, p.q_pos)
    dsa.cache_append(p.dims, p.k_new, p.kv_new, p.table, p.lens, *a, *rows, ws=p.ws)
    dsa.cache_append_rope(p.dims, freq, p.k_new, p.kv_new, p.table, p.lens, *b, *rows, k_offset=-1, kv_offset=-1, ws=p.ws)
    assert dsa.last_launch_count() == 1 and dsa.read_error(p.ws) == 0
    for x, y in zip(a, b):
        assert (x is None and y is None) or torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("mode", ["f32", "bf16"])
@pytest.mark.parametrize("ko,kvo,rot", [(0, -1, 16), (5, 3, 16), (0, 0, 2), (-1, 20, 32)])
def test_append_of_unquantised_rows_is_rope_then_append(mode, ko, kvo, rot):
    p = Append(mode, "act", [300, 1000, 77, 400], [150, 1, 13, 200], 410, **SHAPES[mode])
    a, b = p.caches(), p.caches()
    freq = dsa.rope_frequencies(rot, scaling="yarn", factor=8.0)
    k, kv = p.k_new.clone(), p.kv_new.clone()
    if ko >= 0:
        dsa.rope(k[:, None, ko:ko + rot], freq, q_pos=p.q_pos, layout="half", scale=1.5)
    if kvo >= 0:
        dsa.rope(kv[:, None, kvo:kvo + rot], freq, q_pos=p.q_pos, layout="interleaved", scale=1.5)
    dsa.cache_append(p.dims, k, kv, p.table, p.lens, *a, p.q_seq, p.q_pos, ws=p.ws)
    dsa.cache_append_rope(p.dims, freq, p.k_new, p.kv_new, p.table, p.lens, *b, p.q_seq, p.q_pos, k_offset=ko,
                          kv_offset=kvo, scale=1.5, ws=p.ws)
    assert dsa.read_error(p.ws) == 0
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


def _near_codes(codes, scale, x, mag):
    """codes * scale is x rounded to e4m3 against scale: half a step of 2^-4 of the value (2^-10 below the
    normal range), after the rotation's own error."""
    z = x / scale
    slack = ARITH * mag / scale + 2.0 ** -22 * z.abs()
    ok = (codes - z).abs() <= torch.maximum(z.abs() * 2.0 ** -4, torch.full_like(z, 2.0 ** -10)) + slack
    return bool(ok.all())


@pytest.mark.parametrize("mode,kv", MODES[2:])
@pytest.mark.parametrize("decode", [True, False])
def test_append_of_quantised_rows(mode, kv, decode):
    lens, new = ([1, 63, 64, 65, 128, 500], None) if decode else ([300, 1000, 77, 400], [150, 1, 13, 200])
    p = Append(mode, kv, lens, new, 420)
    s, rot = p.case.spec, 32
    freq = dsa.rope_frequencies(rot)
    before, c = p.caches(), p.caches()
    rows = (None, None) if decode else (p.q_seq, p.q_pos)
    dsa.cache_append_rope(p.dims, freq, p.k_new, p.kv_new, p.table, p.lens, *c, *rows, k_offset=0, k_layout="half", ws=p.ws)
    assert dsa.read_error(p.ws) == 0
    at = p.rows()
    kv64, kvm = p.kv_new.double(), torch.zeros_like(p.kv_new, dtype=torch.float64)
    y, m = rotated64(p.kv_new[:, None, s.d - rot:], p.q_pos, freq, "interleaved")
    kv64[:, s.d - rot:], kvm[:, s.d - rot:] = y[:, 0], m[:, 0]
    k64, km = p.k_new.double(), torch.zeros_like(p.k_new, dtype=torch.float64)
    y, m = rotated64(p.k_new[:, None, :rot], p.q_pos, freq, "half")
    k64[:, :rot], km[:, :rot] = y[:, 0], m[:, 0]
    touched = torch.zeros(p.case.num_blocks * 64, dtype=torch.bool, device="cuda")
    touched[at] = True
    if kv == "fp8":
        rec = dsa.kv_record_bytes(s.d)
        r, old = c[2].view(-1, rec), before[2].view(-1, rec)
        assert torch.equal(r[~touched], old[~touched])
        tiles = (s.d + 127) // 128
        sc = r[at][:, s.d:s.d + 4 * tiles].contiguous().view(torch.float32).double()
        codes = r[at][:, :s.d].contiguous().view(torch.float8_e4m3fn).double()
        assert int(r[at][:, s.d + 4 * tiles:].sum()) == 0
        for j in range(tiles):
            e = slice(128 * j, min(s.d, 128 * j + 128))
            amax = kv64[:, e].abs().amax(1)
            assert bool(((sc[:, j] - amax / 448).abs() <= ARITH * kvm[:, e].amax(1) / 448 + amax / 448 * 2.0 ** -22).all())
            assert _near_codes(codes[:, e], sc[:, j:j + 1], kv64[:, e], kvm[:, e])
    if mode == "mxfp8":
        codes = c[0].view(-1, s.d_I)[at].view(torch.float8_e4m3fn).double()
        X = c[1].view(-1, s.d_I // 32)[at].double() - 127
        top = k64.view(len(at), -1, 32).abs().amax(-1)
        assert bool((torch.floor(torch.log2(top * (1 + 1e-12))) - 8 == X).all())
        sc = torch.exp2(X).repeat_interleave(32, 1)
        z = (k64 / sc).clamp(-448, 448)  # magnitudes in [448, 512) saturate
        assert _near_codes(codes, 1.0, z, km / sc)
        assert torch.equal(c[0].view(-1, s.d_I)[~touched], before[0].view(-1, s.d_I)[~touched])
    if mode == "bf16_kfp8":
        old_sc, new_sc = before[1].double(), c[1].double()
        blocks = torch.unique(at // 64)
        same = torch.ones(p.case.num_blocks, dtype=torch.bool, device="cuda")
        same[blocks] = False
        assert torch.equal(c[1][same], before[1][same]) and torch.equal(c[0][same], before[0][same])
        old = before[0].view(torch.float8_e4m3fn).double() * old_sc[:, None, None]
        want, mag = old.view(-1, s.d_I), torch.zeros_like(old.view(-1, s.d_I))
        want[at], mag[at] = k64, km
        for blk in blocks.tolist():
            n = int((at[at // 64 == blk] % 64).max()) + 1  # the block's tokens; the slots behind are not touched
            x, g = want.view(-1, 64, s.d_I)[blk, :n], mag.view(-1, 64, s.d_I)[blk, :n]
            amax = float(x.abs().max())
            assert abs(float(new_sc[blk]) - amax / 448) <= (ARITH * float(g.max()) + amax * 2.0 ** -22) / 448
            assert _near_codes(c[0][blk, :n].view(torch.float8_e4m3fn).double(), new_sc[blk], x, g)
            assert torch.equal(c[0][blk, n:], before[0][blk, n:])


def test_append_rope_bad_rows_are_skipped_and_reported():
    p = Append("mxfp8", "fp8", [100, 200, 50], [3, 2, 1], 430)
    before, c = p.caches(), p.caches()
    freq = dsa.rope_frequencies(32)
    q_seq, q_pos, table = p.q_seq.clone(), p.q_pos.clone(), p.table.clone()
    q_seq[0] = 99
    q_pos[3] = 10 ** 6
    table[2, 0] = -1
    dsa.cache_append_rope(p.dims, freq, p.k_new, p.kv_new, table, p.lens, *c, q_seq, q_pos, ws=p.ws)
    assert dsa.read_error(p.ws) == 3
    at = p.rows()
    for x, y, w in ((c[0], before[0], p.case.spec.d_I), (c[2], before[2], dsa.kv_record_bytes(p.case.spec.d))):
        x, y = x.view(torch.uint8).view(-1, w), y.view(torch.uint8).view(-1, w)
        diff = (x != y).any(1).nonzero().flatten().tolist()
        assert set(diff) <= {int(at[i]) for i in (1, 2, 4)} and len(diff) == 3


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_frequency_that_is_no_number_gives_nan(dtype, bad):
    """pos * f is no angle then, at position 0 either: its pair is NaN, the other pairs and the rows with a
    negative position are what they are without it."""
    T, H, rot = 5, 3, 64
    freq = dsa.rope_frequencies(rot)
    x = torch.randn((T, H, rot), device="cuda").to(dtype)
    pos = torch.tensor([0, 7, -1, 100000, 3], dtype=torch.int32, device="cuda")
    for layout, cols in (("interleaved", [10, 11]), ("half", [5, 37])):
        want = dsa.rope(x, freq, q_pos=pos, layout=layout, out=torch.empty_like(x))
        f = freq.clone()
        f[5] = bad
        got = dsa.rope(x, f, q_pos=pos, layout=layout, out=torch.empty_like(x))
        turned = pos >= 0
        assert got[turned][..., cols].isnan().all() and torch.equal(got[~turned], x[~turned])
        rest = [c for c in range(rot) if c not in cols]
        assert torch.equal(got[..., rest], want[..., rest])


def test_append_with_a_frequency_that_is_no_number_writes_nan():
    p = Append("bf16", "act", [100, 200], [3, 2], 440)
    s, rot = p.case.spec, 16
    a, b = p.caches(), p.caches()
    freq = dsa.rope_frequencies(rot)
    f = freq.clone()
    f[2] = math.inf
    for c, g in ((a, freq), (b, f)):
        dsa.cache_append_rope(p.dims, g, p.k_new, p.kv_new, p.table, p.lens, *c, p.q_seq, p.q_pos, ws=p.ws)
    assert dsa.read_error(p.ws) == 0
    at = p.rows()
    for x, y, w, cols in ((a[0], b[0], s.d_I, [2, 2 + rot // 2]), (a[2], b[2], s.d, [s.d - rot + 4, s.d - rot + 5])):
        x, y = x.view(-1, w)[at], y.view(-1, w)[at]
        assert y[:, cols].isnan().all()
        rest = [c for c in range(w) if c not in cols]
        assert torch.equal(x[:, rest], y[:, rest])


class Turn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, freq, pos, layout):
        ctx.save_for_backward(freq, pos)
        ctx.layout = layout
        return dsa.rope(x, freq, q_pos=pos, layout=layout, out=torch.empty_like(x), scale=0.7)

    @staticmethod
    def backward(ctx, dy):
        freq, pos = ctx.saved_tensors
        return dsa.rope(dy, freq, q_pos=pos, layout=ctx.layout, out=torch.empty_like(dy), scale=0.7, transpose=True), None, None, None


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_gradients_come_from_a_function_of_the_callers_and_are_not_lost(layout):
    T, H, rot = 9, 4, 32
    freq = dsa.rope_frequencies(rot)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 771
    x, dy = torch.randn((T, H, rot), device="cuda", requires_grad=True), torch.randn((T, H, rot), device="cuda")
    Turn.apply(x, freq, pos, layout).backward(dy)
    check(x.grad, dy, pos, freq, layout, 0.7, True)
    with pytest.raises(ValueError, match="gradient"):
        dsa.rope(x, freq, q_pos=pos, layout=layout, out=torch.empty_like(dy))
    with torch.no_grad():
        check(dsa.rope(x, freq, q_pos=pos, layout=layout, out=torch.empty_like(dy)), x.detach(), pos, freq, layout)


def test_what_is_written_in_place_counts_as_changed():
    """A tensor that autograd keeps for a backward pass and that one of these calls then overwrites is an error in
    that pass, as with any operation in place: its gradient would be formed from the new values."""
    def changed(t, call):
        w = torch.ones((), device="cuda", requires_grad=True)
        y = (w * t).sum()
        call()
        with pytest.raises(RuntimeError, match="inplace operation"):
            y.backward()

    freq, pos = dsa.rope_frequencies(16), torch.arange(6, dtype=torch.int32, device="cuda")
    x, a, b = (torch.randn((6, 2, 48), device="cuda") for _ in range(3))
    changed(x, lambda: dsa.rope(x[..., :16], freq, q_pos=pos))
    changed(b, lambda: dsa.rope([x[..., :16], a[..., :16]], freq, q_pos=pos, out=[a[..., 16:32], b[..., 32:]]))
    p = Append("bf16", "act", [100, 200], [3, 2], 450)
    k, _, kv = p.caches()
    s = p.case.spec
    k_out, kv_out = torch.empty((300, s.d_I), device="cuda").bfloat16(), torch.empty((300, s.d), device="cuda").bfloat16()
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    read = lambda: dsa.cache_read(p.dims, k, None, kv, p.table, p.lens, cu, 300, k_out=k_out, kv_out=kv_out, ws=p.ws)  # noqa: E731
    changed(k_out, read)
    changed(kv_out, read)
    q = torch.randn((6, 2, 16), device="cuda")
    dims = dsa.prompt_dims(q, q, q, 1)
    ws, out, lse = dsa.prompt_workspace(dims, 6), torch.empty_like(q), torch.empty((6, 2), device="cuda")
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    attend = lambda: dsa.prompt_attn(dims, q, q, q, cu, cu, 0.25, ws=ws, out=out, lse=lse)  # noqa: E731
    changed(out, attend)
    changed(lse, attend)
    with torch.inference_mode():  # tensors without a count of changes
        y = torch.randn((6, 2, 16), device="cuda")
        assert dsa.rope(y, freq, q_pos=pos) is y
    assert dsa.read_error(p.ws) == 0 and dsa.read_error(ws) == 0


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("lo,hi", [(0, 1 << 12), (1 << 12, 1 << 20), ((1 << 31) - 5000, 1 << 31)])
def test_rope_error_of_near_and_far_positions(layout, lo, hi):
    """fp32: cos and sin within two steps (2^-23; one is what the function promises), their correction rounds by
    2^-25, the products with the scale and with an element by 2^-24 each, the sum by half a step of the result.
    The angle is off by the cut of the frequency's turns, 2 pi 2^-33, and by fp64's roundings of the frequency in
    turns (two, 2^-52 of the angle) and, in the definition, of the product (2^-53)."""
    T, H, rot = 300, 4, 64
    g = torch.Generator(device="cuda").manual_seed(lo % 1000 + 7)
    x = torch.randn((T, H, rot), generator=g, device="cuda")
    pos = torch.randint(lo, hi, (T,), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    freq = dsa.rope_frequencies(rot)
    y = dsa.rope(x, freq, q_pos=pos, layout=layout, out=torch.empty_like(x), scale=1.25)
    want, mag = rotated64(x, pos, freq, layout, 1.25)
    angle = pos.double()[:, None] * freq
    angle = torch.cat((angle, angle), -1) if layout == "half" else angle.repeat_interleave(2, -1)
    arith = 4.5 * 2.0 ** -24 + 2 * math.pi * 2.0 ** -33 + 1.5 * 2.0 ** -52 * angle[:, None]
    tol = want.abs() * 2.0 ** -24 + 1.25 * arith * mag * (1 + 2.0 ** -24)
    assert bool(((y.double() - want).abs() <= tol * (1 + 2.0 ** -7)).all()), float(((y.double() - want).abs() / tol).max())


@pytest.mark.parametrize("dtype,rot,layout", [(torch.bfloat16, 16, "half"), (torch.bfloat16, 8, "interleaved"), (torch.float32, 8, "half"),
                                              (torch.float32, 4, "interleaved")])
def test_rope_of_heads_of_one_piece(dtype, rot, layout):
    """Aligned heads whose columns, or halves of them, fill just 16 bytes; alone and as part of wider heads."""
    T, H = 50, 5
    freq = dsa.rope_frequencies(rot)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 313
    wide = torch.randn((T, H, 3 * rot), device="cuda").to(dtype)
    for x in (wide[..., :rot].contiguous(), wide[..., rot:2 * rot]):
        keep = x.clone()
        check(dsa.rope(x, freq, q_pos=pos, layout=layout, out=torch.empty_like(keep)), keep, pos, freq, layout)
        check(dsa.rope(x, freq, q_pos=pos, layout=layout), keep, pos, freq, layout)
