"""dsa_prompt_attn against softmax attention in 64 bits: packed lengths from none to many tiles, grouped heads,
widths that fill no tile, prefixes, queries without keys, strided views, garbage behind the packed rows."""
import math

import pytest
import torch

import indexer_top_sparse_paged_gb300 as dsa

pytestmark = pytest.mark.gpu


def starts(n):
    return torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def reference(q, k, v, nq, nk, scale, causal):
    """(out, lse, sum p |v|, largest sum |q||k|) in fp64."""
    H, G = q.shape[1], q.shape[1] // k.shape[1]
    out = torch.zeros((q.shape[0], H, v.shape[2]), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    lse = torch.full((q.shape[0], H), -math.inf, dtype=torch.float64, device="cuda")
    zmag = torch.zeros_like(lse)
    a = b = 0
    for n, m in zip(nq, nk):
        if n and m:
            Q = q[a:a + n].double().transpose(0, 1)
            K = k[b:b + m].double().transpose(0, 1).repeat_interleave(G, 0)
            V = v[b:b + m].double().transpose(0, 1).repeat_interleave(G, 0)
            z = Q @ K.transpose(1, 2) * scale
            if causal:
                z = z.masked_fill(torch.ones((n, m), dtype=torch.bool, device="cuda").triu(m - n + 1), -math.inf)
            e = torch.logsumexp(z, -1)
            p = torch.exp(z - torch.where(e == -math.inf, torch.zeros_like(e), e)[..., None])
            out[a:a + n], mag[a:a + n] = (p @ V).transpose(0, 1), (p @ V.abs()).transpose(0, 1)
            lse[a:a + n] = e.T
            zmag[a:a + n] = (Q.abs() @ K.abs().transpose(1, 2)).amax(-1).T * scale
        a, b = a + n, b + m
    return out, lse, mag, zmag


def check(got, q, k, v, nq, nk, scale, causal=True):
    out, lse = got
    n = sum(nq)
    o, e, mag, zmag = reference(q[:n], k, v, nq, nk, scale, causal)
    d = q.shape[2]
    # logits: an fp32 sum of d products rounds d + 2 times at most; a weight follows by that and three
    # roundings of the exponential; sums over the keys add one rounding a key
    zerr = (d + 2) * 2.0 ** -24 * zmag + 2.0 ** -22 * (1 + e.abs().nan_to_num(posinf=0.0))
    keys = max(nk, default=0)
    half = 2.0 ** -8 if q.dtype == torch.bfloat16 else 0.0  # the weights and the output in bf16: half a step each
    tol = (2 * zerr[..., None] + half + (keys + 8) * 2.0 ** -24) * mag * 1.01 + (half or 2.0 ** -23) * o.abs() * 1.01
    assert torch.equal(torch.isinf(lse[:n]), torch.isinf(e)) and not lse[:n].isnan().any()
    live = ~torch.isinf(e)
    assert bool(((lse[:n].double() - e).abs()[live] <= (zerr + (keys + 8) * 2.0 ** -24)[live]).all()), \
        float((lse[:n].double() - e).abs()[live].max())
    err = (out[:n].double() - o).abs()
    assert not out[:n].isnan().any() and bool((err <= tol + 1e-30).all()), (float((err - tol).max()), int((err > tol).sum()))
    assert not out[:n][~live].any()


def make(dtype, nq, nk, H, H_kv, d_qk, d_v, seed=0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    q, k, v = r(sum(nq) + pad, H, d_qk), r(sum(nk) + pad, H_kv, d_qk), r(sum(nk) + pad, H_kv, d_v)
    if pad:  # rows behind the last sequence hold anything
        for t, n in ((q, nq), (k, nk), (v, nk)):
            t[sum(n):] = float("nan")
    return q, k, v


def attend(q, k, v, nq, nk, scale, causal=True, **kw):
    dims = dsa.prompt_dims(q, k, v, len(nq), causal)
    ws = dsa.prompt_workspace(dims, q.shape[0])
    got = dsa.prompt_attn(dims, q, k, v, starts(nq), starts(nk), scale, ws=ws, **kw)
    assert dsa.read_error(ws) == 0
    return got


LENS = [([1], None), ([64], None), ([65, 1, 0, 63], None), ([127, 128, 129], None), ([0, 0, 5, 0], None), ([300, 1, 0, 700], None),
        ([1, 1, 1], [1, 200, 1025]), ([33, 257], [500, 257]), ([40, 7, 300], [10, 0, 299]), ([257], [511])]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("nq,nk", LENS)
@pytest.mark.parametrize("causal", [True, False])
def test_packed_lengths(dtype, nq, nk, causal):
    nk = nq if nk is None else nk
    q, k, v = make(dtype, nq, nk, 8, 2, 128, 128, seed=len(nq), pad=9)
    check(attend(q, k, v, nq, nk, 128 ** -0.5, causal), q, k, v, nq, nk, 128 ** -0.5, causal)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,H_kv", [(1, 1), (7, 1), (12, 4), (6, 6), (64, 8), (130, 1), (24, 8)])
def test_grouped_heads(dtype, H, H_kv):
    nq, nk = [70, 1, 19], [70, 333, 150]
    q, k, v = make(dtype, nq, nk, H, H_kv, 64, 64, seed=H)
    check(attend(q, k, v, nq, nk, 0.125), q, k, v, nq, nk, 0.125)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d_qk,d_v", [(192, 128), (8, 8), (80, 72), (96, 96), (64, 128), (128, 64), (256, 256), (200, 136), (72, 256)])
def test_widths(dtype, d_qk, d_v):
    nq, nk = [150, 3, 129], [150, 400, 300]
    q, k, v = make(dtype, nq, nk, 4, 2, d_qk, d_v, seed=d_qk)
    check(attend(q, k, v, nq, nk, d_qk ** -0.5), q, k, v, nq, nk, d_qk ** -0.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_longer_prompts(dtype):
    for nq, nk, H, H_kv, d_qk, d_v in (([1500, 900], [1500, 2100], 4, 4, 192, 128), ([1], [20000], 8, 1, 128, 128),
                                       ([1] * 40, list(range(1, 4000, 100)), 8, 2, 128, 128), ([2500], [2500], 2, 1, 128, 128)):
        q, k, v = make(dtype, nq, nk, H, H_kv, d_qk, d_v, seed=H)
        check(attend(q, k, v, nq, nk, d_qk ** -0.5), q, k, v, nq, nk, d_qk ** -0.5)


def test_many_short_sequences():
    """Several units a CTA, most of them with one short query tile, some with no keys: every one in turn."""
    nq = [100, 1, 128, 129, 3, 0, 256, 257, 40] * 9
    nk = [max(0, n - 7) if i % 4 == 0 else n + 5 * (i % 3) for i, n in enumerate(nq)]
    q, k, v = make(torch.bfloat16, nq, nk, 16, 16, 192, 128, seed=11, pad=3)
    check(attend(q, k, v, nq, nk, 192 ** -0.5), q, k, v, nq, nk, 192 ** -0.5)
    nq = [1] * 1500  # more sequences than the plan looks at in one go
    nk = [i % 5 for i in range(1500)]
    q, k, v = make(torch.bfloat16, nq, nk, 4, 2, 64, 64, seed=12)
    check(attend(q, k, v, nq, nk, 0.125), q, k, v, nq, nk, 0.125)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_and_growing_logits(dtype):
    """Scores that grow along the keys move every row's running maximum in every tile; then a few huge ones."""
    nq = nk = [700]
    q, k, v = make(dtype, nq, nk, 2, 1, 64, 64, seed=3)
    k *= torch.linspace(0.1, 12.0, 700, device="cuda")[:, None, None].to(dtype)
    check(attend(q, k, v, nq, nk, 0.5), q, k, v, nq, nk, 0.5)
    q.mul_(64)
    check(attend(q, k, v, nq, nk, 0.5), q, k, v, nq, nk, 0.5)
    z = torch.zeros_like(q)
    out, lse = attend(z, k, v, nq, nk, 0.5)  # equal logits: the mean of the values seen
    check((out, lse), z, k, v, nq, nk, 0.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_views_and_rows_left_alone(dtype):
    """q and k, v as parts of wider projections; out and lse behind the last sequence stay as they were."""
    nq, nk, H = [130, 60], [130, 260], 4
    wide = torch.randn((sum(nq) + 5, H, 320), device="cuda").to(dtype)
    kv = torch.randn((H, sum(nk), 320), device="cuda").to(dtype).transpose(0, 1)
    q, k, v = wide[..., 64:256], kv[..., :192], kv[..., 192:]
    out = torch.full((len(wide), H, 128), 3.0, dtype=dtype, device="cuda")
    lse = torch.full((len(wide), H), 3.0, device="cuda")
    got = attend(q, k, v, nq, nk, 192 ** -0.5, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    check(got, q, k, v, nq, nk, 192 ** -0.5)
    assert bool((out[sum(nq):] == 3).all()) and bool((lse[sum(nq):] == 3).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_key_head_expanded_over_all(dtype):
    """Key heads that are one stored head (stride 0), alone and together with one value row for all keys."""
    nq, nk = [130, 7], [130, 300]
    q, k, v = make(dtype, nq, nk, 6, 1, 128, 64, seed=21)
    k, v = k.expand(-1, 3, -1), v.expand(-1, 3, -1)
    check(attend(q, k, v, nq, nk, 0.1), q, k, v, nq, nk, 0.1)
    v = v[:1].expand(len(v), -1, -1)
    check(attend(q, k, v, nq, nk, 0.1), q, k, v, nq, nk, 0.1)
    q = q[:, :1].expand(-1, 6, -1)
    check(attend(q, k, v, nq, nk, 0.1), q, k, v, nq, nk, 0.1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_workspace_serves_smaller_calls_and_the_least_size_does(dtype):
    """The size grows with the query tokens, and a call with just that many bytes is not refused and writes no
    byte behind them: long single tokens split their keys over every partial there is room for."""
    for B, H, H_kv, L in ((1, 8, 1, 9000), (3, 64, 8, 5000), (40, 8, 2, 700), (5, 130, 130, 600)):
        nq, nk = [1] * B, [L - 13 * i for i in range(B)]
        q, k, v = make(dtype, nq, nk, H, H_kv, 64, 64, seed=B)
        dims = dsa.prompt_dims(q, k, v, B)
        sizes = [dsa.prompt_workspace(dims, n).numel() for n in (0, 1, B, 4 * B, 4 * B + 1, 300, 5000)]
        assert sizes == sorted(sizes)
        n = sizes[2]
        room = torch.full((n + 4096 + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        off = -room.data_ptr() % 256
        ws = room[off:off + n]
        ws[:256] = 0
        got = dsa.prompt_attn(dims, q, k, v, starts(nq), starts(nk), 0.125, ws=ws)
        check(got, q, k, v, nq, nk, 0.125)
        assert dsa.read_error(ws) == 0 and bool((room[off + n:] == 0x5A).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_calls_around_the_one_launch_form(dtype):
    """32 and 33 sequences, 896 and 897 keys in all, as many units as CTAs and more: the same answers with and
    without a work list."""
    for nq, nk, H, H_kv in (([3] * 32, [28] * 32, 4, 2), ([3] * 33, [27] * 33, 4, 2), ([100], [896], 2, 2), ([100], [897], 2, 2),
                            ([1], [896], 130, 130), ([5], [300], 152, 152), ([5], [300], 153, 153), ([1] * 8, [112] * 8, 19, 19),
                            ([0, 0, 4], [0, 9, 4], 3, 1), ([896], [896], 19, 19)):
        q, k, v = make(dtype, nq, nk, H, H_kv, 64, 64, seed=H)
        check(attend(q, k, v, nq, nk, 0.125), q, k, v, nq, nk, 0.125)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bad_offsets_are_skipped_and_reported(dtype):
    q, k, v = make(dtype, [100], [100], 4, 2, 64, 64)
    dims = dsa.prompt_dims(q, k, v, 3)
    ws = dsa.prompt_workspace(dims, 100)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for cu_q, cu_k, bad in ((i32(0, 40, 30, 60), i32(0, 40, 60, 90), slice(30, 40)), (i32(0, 20, 60, 101), i32(0, 20, 60, 90), slice(60, 100)),
                            (i32(0, 20, 60, 90), i32(0, 20, 60, 101), slice(60, 90))):
        out = torch.full((100, 4, 64), 3.0, dtype=dtype, device="cuda")
        dsa.prompt_attn(dims, q, k, v, cu_q, cu_k, 0.125, ws=ws, out=out)
        assert dsa.read_error(ws) == 2
        if bad.start >= 60:
            assert bool((out[bad] == 3).all())
            again = attend(q[:60], k[:60], v[:60], [20, 40], [20, 40], 0.125)
            assert torch.equal(again[0], out[:60])


def test_streams_graphs_and_repeated_calls():
    nq, nk = [300, 1, 77], [300, 900, 500]
    q, k, v = make(torch.bfloat16, nq, nk, 8, 2, 128, 128)
    scale = 128 ** -0.5
    first = attend(q, k, v, nq, nk, scale)
    dims = dsa.prompt_dims(q, k, v, 3)
    ws = [dsa.prompt_workspace(dims, q.shape[0]) for _ in range(2)]
    cu_q, cu_k = starts(nq), starts(nk)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for i in range(6):  # two streams at once, each with its workspace
        got.append(dsa.prompt_attn(dims, q, k, v, cu_q, cu_k, scale, ws=ws[i % 2], stream=streams[i % 2]))
    torch.cuda.synchronize()
    for o, e in got:  # the same bits every time
        assert torch.equal(o, first[0]) and torch.equal(e, first[1])
    out, lse = torch.zeros_like(first[0]), torch.zeros_like(first[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.prompt_attn(dims, q, k, v, cu_q, cu_k, scale, ws=ws[0], out=out, lse=lse)
    cu_q.copy_(starts([10, 300, 68]))
    cu_k.copy_(starts([500, 300, 900]))
    q.normal_()
    for _ in range(2):
        g.replay()
    check((out, lse), q, k, v, [10, 300, 68], [500, 300, 900], scale)
    assert dsa.read_error(ws[0]) == 0


def test_empty_calls_launch_nothing():
    q, k, v = make(torch.bfloat16, [0], [5], 4, 2, 64, 64)
    dims = dsa.prompt_dims(q, k, v, 1)
    ws = dsa.prompt_workspace(dims, 0)
    out, lse = dsa.prompt_attn(dims, q, k, v, starts([0]), starts([5]), 0.125, ws=ws)
    assert out.shape == (0, 4, 64) and dsa.last_launch_count() == 0
    q, k, v = make(torch.bfloat16, [6], [0], 4, 2, 64, 64)  # queries, and no keys anywhere
    check(attend(q, k, v, [6], [0], 0.125), q, k, v, [6], [0], 0.125)


def test_a_prompt_step_around_the_decode_step():
    """The operators in the order a step uses them, in fp32: rotate, append, read the prefix back, project it up
    and attend over the prompt; the decode step's attention over every selected position gives the same answer
    through the absorbed query (q W_k) and the absorbed value projection."""
    torch.manual_seed(5)
    L, H, nope, rope, r, dv, K = 200, 4, 32, 16, 64, 32, 256
    d, d_I, H_I = r + rope, 32, 2
    blocks = (L + 63) // 64
    dims = dsa.make_dims("f32", 1, blocks, blocks, H_I, d_I, H, d, r, K)
    ws = dsa.workspace(dims, L)
    table = torch.randperm(blocks, device="cuda").to(torch.int32)[None].contiguous()
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    pos, seq = torch.arange(L, dtype=torch.int32, device="cuda"), torch.zeros(L, dtype=torch.int32, device="cuda")
    freq = dsa.rope_frequencies(rope)
    lat, k_I = torch.randn((L, d), device="cuda"), torch.randn((L, d_I), device="cuda")
    Wk, Wv = torch.randn((H, r, nope), device="cuda") * r ** -0.5, torch.randn((H, r, dv), device="cuda") * r ** -0.5
    q = torch.randn((L, H, nope + rope), device="cuda")
    scale = (nope + rope) ** -0.5
    dsa.rope(q[..., nope:], freq, q_pos=pos)
    kc, kvc = torch.zeros((blocks, 64, d_I), device="cuda"), torch.zeros((blocks, 64, d), device="cuda")
    dsa.cache_append_rope(dims, freq, k_I, lat, table, lens, kc, None, kvc, seq, pos, ws=ws)
    k_back, kv_back = dsa.cache_read(dims, kc, None, kvc, table, lens, torch.tensor([0, L], dtype=torch.int32, device="cuda"), L, ws=ws)
    k = torch.cat((torch.einsum("tr,hrn->thn", kv_back[:, :r], Wk), kv_back[:, None, r:].expand(L, H, rope)), -1)
    v = torch.einsum("tr,hrv->thv", kv_back[:, :r], Wv)
    out, lse = attend(q, k, v, [L], [L], scale)
    check((out, lse), q, k, v, [L], [L], scale)
    # absorbed: q' = [W_k q_nope, q_rope] over the latent rows themselves, the causal positions as the selection
    qa = torch.cat((torch.einsum("thn,hrn->thr", q[..., :nope], Wk), q[..., nope:]), -1).contiguous()
    idx = torch.arange(K, device="cuda", dtype=torch.int32)[None].expand(L, K)
    idx = torch.where(idx <= pos[:, None], idx, torch.full_like(idx, -1)).contiguous()
    o, e = dsa.sparse_attn(dims, qa, kvc, table, lens, idx, scale, q_seq=seq, ws=ws)
    assert dsa.read_error(ws) == 0
    o = torch.einsum("thr,hrv->thv", o, Wv)
    # two orders of the same fp32 products, of order 1, through at most d + r + dv roundings each
    assert float((o - out).abs().max()) <= 2 * (d + r + dv) * 2.0 ** -24 * 32
    assert float((e - lse).abs().max()) <= 2 * (d + r + dv) * 2.0 ** -24 * 32


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_overlapping_sequences_fit_the_lists(dtype):
    """Entries that descend every other time leave 300 sequences over the same rows, with far more row tiles
    than the lists were made for: reported, the rows either right or left as they were, and the workspace
    good for the next call."""
    n, m, B = 3000, 70, 600
    q, k, v = make(dtype, [n], [m], 4, 1, 64, 64)
    dims = dsa.prompt_dims(q, k, v, B, False)
    ws = dsa.prompt_workspace(dims, n)
    cu_q = torch.tensor([0, n], dtype=torch.int32, device="cuda").repeat(B // 2 + 1)[: B + 1].contiguous()
    cu_k = torch.tensor([0, m], dtype=torch.int32, device="cuda").repeat(B // 2 + 1)[: B + 1].contiguous()
    out = torch.full((n, 4, 64), 9.0, dtype=dtype, device="cuda")
    got, _ = dsa.prompt_attn(dims, q, k, v, cu_q, cu_k, 0.125, ws=ws, out=out)
    assert dsa.read_error(ws) == 2
    want, _ = attend(q, k, v, [n], [m], 0.125, causal=False)
    left = (got == 9.0).all(-1)
    assert torch.equal(got[~left], want[~left]) and not left.all()
    nq, nk = [n] + [0] * (B - 1), [m] + [0] * (B - 1)
    got = dsa.prompt_attn(dims, q, k, v, starts(nq), starts(nk), 0.125, ws=ws)
    assert dsa.read_error(ws) == 0
    check(got, q, k, v, nq, nk, 0.125, causal=False)


@pytest.mark.parametrize("dtype,d_qk,d_v", [(torch.float32, 20, 12), (torch.float32, 64, 68), (torch.bfloat16, 72, 88),
                                            (torch.bfloat16, 200, 24)])
@pytest.mark.parametrize("nq,nk", [([1, 1, 1], [5000, 1, 2100]), ([96], [6000]), ([300], [4000])])
def test_split_keys_of_odd_widths(dtype, d_qk, d_v, nq, nk):
    """Rows whose keys are split and joined where the last columns fill no run of eight or sixteen."""
    q, k, v = make(dtype, nq, nk, 6, 2, d_qk, d_v, seed=d_v, pad=3)
    check(attend(q, k, v, nq, nk, d_qk ** -0.5), q, k, v, nq, nk, d_qk ** -0.5)


def test_many_units_of_mixed_lengths():
    """Far more units than CTAs, long ones, short ones and ones without keys in turn."""
    nq = [700, 1, 130, 0, 129, 300, 40] * 6
    nk = [900, 3000, 130, 64, 0, 300, 20] * 6
    q, k, v = make(torch.bfloat16, nq, nk, 32, 8, 64, 64, seed=3, pad=5)
    check(attend(q, k, v, nq, nk, 0.125), q, k, v, nq, nk, 0.125)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 200])
def test_a_row_of_nan_stays_nan_whether_its_keys_are_split_or_not(dtype, d):
    """A query that is NaN has no logit that compares, in no part of its keys: its row is NaN all the same, in
    one pass over the keys and joined from many, and the other rows are what they are without it."""
    for nq, nk in (([3, 2], [40, 300]), ([1, 2, 1], [9000, 6000, 700])):
        q, k, v = make(dtype, nq, nk, 8, 2, d, d, seed=31)
        clean = attend(q, k, v, nq, nk, d ** -0.5)
        row, head = nq[0], 5  # the second sequence's first query
        q[row, head] = float("nan")
        out, lse = attend(q, k, v, nq, nk, d ** -0.5)
        assert out[row, head].isnan().all() and lse[row, head].isnan()
        rest = torch.ones(lse.shape, dtype=torch.bool, device="cuda")
        rest[row, head] = False
        assert torch.equal(out[rest], clean[0][rest]) and torch.equal(lse[rest], clean[1][rest])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("nq,nk", [([40, 50, 30], [40, 50, 30]), ([40, 50, 30], [500, 300, 2000]), ([2] * 40, [30] * 40)])
def test_bad_sequences_between_good_ones(dtype, nq, nk):
    """A sequence whose bounds descend or leave the tensors, in calls with and without a work list (more than 896
    keys, more than 32 sequences): reported; the good sequences around it are right, and the rows of the bad one
    and those behind the last one stay as they were."""
    B, spare = len(nq), 20
    q, k, v = (t.nan_to_num() for t in make(dtype, nq, nk, 8, 2, 64, 64, seed=B, pad=spare))
    dims = dsa.prompt_dims(q, k, v, B)
    ws = dsa.prompt_workspace(dims, len(q))
    for which in ("queries descend", "keys descend", "queries leave", "keys leave"):
        cu_q, cu_k = starts(nq).tolist(), starts(nk).tolist()
        cu, n = (cu_q, len(q)) if which.startswith("queries") else (cu_k, len(k))
        if which.endswith("descend"):  # sequence 1 ends before it starts; sequence 2 begins there
            cu[2] = cu[1] - 1
        else:
            cu[-1] = n + 1
        bad = 1 if which.endswith("descend") else B - 1
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        out, lse = torch.full((len(q), 8, 64), 3.0, dtype=dtype, device="cuda"), torch.full((len(q), 8), 3.0, device="cuda")
        dsa.prompt_attn(dims, q, k, v, i32(cu_q), i32(cu_k), 0.125, ws=ws, out=out, lse=lse)
        assert dsa.read_error(ws) == 2
        untouched = torch.ones(len(q), dtype=torch.bool, device="cuda")
        for b in range(B):
            if b == bad:
                continue
            a, e = cu_q[b], cu_q[b + 1]
            untouched[a:e] = False
            # a row that two sequences claim has the answer of either: leave it out (the rest are the last positions still)
            a, e = a + (which == "queries descend" and b == 2), e - (which == "queries descend" and b == 0)
            ka, ke = cu_k[b], cu_k[b + 1] - (which == "queries descend" and b == 0)
            check((out[a:e], lse[a:e]), q[a:e], k[ka:ke], v[ka:ke], [e - a], [ke - ka], 0.125)
        assert bool((out[untouched] == 3).all()) and bool((lse[untouched] == 3).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,H_kv", [(8, 2), (6, 2), (4, 4)])
def test_orders_of_heads_and_tokens(dtype, H, H_kv):
    """Queries stored head by head, keys and values token by token and the other way round; token strides that are
    no multiple of the head's; keys whose rows overlap in memory."""
    nq, nk, d = [130, 1, 64], [130, 900, 300], 64
    q, k, v = make(dtype, nq, nk, H, H_kv, d, d, seed=H)
    want = attend(q, k, v, nq, nk, 0.125)
    check(want, q, k, v, nq, nk, 0.125)
    by_head = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731

    def padded(t, extra):
        room = torch.full((t.shape[0], t.shape[1] * t.shape[2] + extra), float("nan"), device="cuda").to(dtype)
        view = room[:, :t.shape[1] * t.shape[2]].unflatten(1, t.shape[1:])
        view.copy_(t)
        return view

    for a, b, c in ((by_head(q), k, v), (by_head(q), by_head(k), v), (q, k, by_head(v)), (padded(q, 8), padded(k, 24), padded(v, 40)),
                    (by_head(q), padded(k, 8), by_head(v)), (padded(q, 72), by_head(k), padded(v, 8))):
        got = attend(a, b, c, nq, nk, 0.125)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    line = torch.randn((sum(nk) * 8 + 64 * H_kv,), device="cuda").to(dtype)
    k = line.as_strided((sum(nk), H_kv, d), (8, d, 1))  # each key starts 8 elements after the one before
    check(attend(q, k, v, nq, nk, 0.125), q, k, v, nq, nk, 0.125)
