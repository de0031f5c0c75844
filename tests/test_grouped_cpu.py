"""Refusals of the grouped-head calls, before anything is launched (no GPU needed)."""
import ctypes
import math
import random

import pytest
import torch

import indexer_top_sparse_paged_gb300 as dsa
from indexer_top_sparse_paged_gb300.build import build_library

FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: every call below fails its checks first
FAKE2 = ctypes.c_void_p(1 << 21)
ODD = ctypes.c_void_p((1 << 20) + 4)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    build_library()
    return dsa.lib()


def _dims(**kw):
    d = dict(type="bf16", B=2, max_blocks=4, num_blocks=8, H=8, H_kv=2, d_qk=128, d_v=128, block_size=64)
    d.update(kw)
    return dsa.grouped_dims(**d)


def _raw(**kw):
    d = _dims()
    for n, v in kw.items():
        setattr(d, n, v)
    return d


BAD_DIMS = [(dict(type=2), 2), (dict(type=-1), 2), (dict(block_size=32), 2), (dict(B=0), 1), (dict(max_blocks=0), 1), (dict(num_blocks=0), 1),
            (dict(H=0), 1), (dict(H_kv=0), 1), (dict(H=7), 1), (dict(d_qk=0), 1), (dict(d_v=-16), 1), (dict(d_qk=272), 2), (dict(d_v=264), 2),
            (dict(d_qk=72), 2), (dict(d_v=8), 2), (dict(num_blocks=1 << 25), 2), (dict(max_blocks=1 << 25), 2),
            (dict(H=40000, H_kv=40000, num_blocks=1), 2)]


def test_dims(L):
    size = lambda d, T=2, w=0: L.dsa_grouped_workspace_size(ctypes.byref(d), T, w)  # noqa: E731
    assert L.dsa_grouped_workspace_size(None, 2, 0) == 0 and size(_dims(), -1) == 0 and size(_dims(), 1 << 29) == 0
    assert 0 < size(_dims()) < size(_dims(), 2, 1)
    assert size(_dims(), 4) >= size(_dims(), 2) and size(_dims(), 4, 1) >= size(_dims(), 2, 1)
    for kw, st in BAD_DIMS:
        d = _raw(**kw)
        assert size(d) == 0, kw
        assert _append(L, d) == st and _attn(L, d) == st and _evict(L, d) == st, kw
    with pytest.raises(ValueError, match="type"):
        _dims(type="fp16")


def _append(L, dims=None, k=FAKE, ks=(256, 128), v=FAKE, vs=(256, 128), table=FAKE, lens=FAKE, cu=None, T=2, kc=FAKE, sc=FAKE, vc=FAKE,
            vsc=FAKE, ws=FAKE, nbytes=BIG):
    return L.dsa_grouped_append(dims or _dims(), k, *ks, v, *vs, table, lens, cu, T, kc, sc, vc, vsc, ws, nbytes, None)


def test_append_refusals(L):
    assert _append(L, cu=FAKE, T=0) == 0 and L.dsa_last_launch_count() == 0
    for name in ("k", "v", "table", "lens", "kc", "sc", "vc", "vsc"):
        assert _append(L, **{name: None}) == 1, name
    for name in ("k", "v", "kc", "vc"):
        assert _append(L, **{name: ODD}) == 1, name
    for bad in ((-256, 128), (256, -128), (257, 128), (256, 4), (1 << 40, 128)):
        assert _append(L, ks=bad) == 1 and _append(L, vs=bad) == 1, bad
    assert _append(L, T=3) == 1 and _append(L, T=-1, cu=FAKE) == 1
    assert _append(L, ws=None) == 3 and _append(L, ws=ODD) == 3 and _append(L, nbytes=255) == 3
    assert L.dsa_grouped_append(None, FAKE, 256, 128, FAKE, 256, 128, FAKE, FAKE, None, 2, FAKE, FAKE, FAKE, FAKE, FAKE, BIG, None) == 1


def _attn(L, dims=None, q=FAKE, qs=(1024, 128), kc=FAKE, sc=FAKE, vc=FAKE, vsc=FAKE, table=FAKE, lens=FAKE, cu=None, T=2, scale=0.1, out=FAKE,
          lse=None, w=None, wo=None, ws=FAKE, nbytes=BIG):
    return L.dsa_grouped_attn(dims or _dims(), q, *qs, kc, sc, vc, vsc, table, lens, cu, T, scale, out, lse, w, wo, ws, nbytes, None)


def test_attn_refusals(L):
    assert _attn(L, cu=FAKE, T=0) == 0 and L.dsa_last_launch_count() == 0
    for name in ("q", "kc", "sc", "vc", "vsc", "table", "lens", "out"):
        assert _attn(L, **{name: None}) == 1, name
    for name in ("q", "kc", "vc", "out"):
        assert _attn(L, **{name: ODD}) == 1, name
    for bad in ((-1024, 128), (1024, -128), (1025, 128), (1024, 4), (1 << 40, 128)):
        assert _attn(L, qs=bad) == 1, bad
    for s in (0.0, -1.0, math.nan, math.inf):
        assert _attn(L, scale=s) == 1
    assert _attn(L, T=3) == 1 and _attn(L, T=-1, cu=FAKE) == 1 and _attn(L, T=1 << 29, cu=FAKE) == 2
    assert _attn(L, w=FAKE) == 1  # weights to add to, and nowhere to write them
    d = _dims()
    for w in (None, FAKE2):
        need = L.dsa_grouped_workspace_size(d, 2, w is not None)
        assert _attn(L, ws=None, wo=w) == 3 and _attn(L, ws=ODD, wo=w) == 3 and _attn(L, nbytes=need - 1, wo=w) == 3


def _evict(L, dims=None, w=FAKE, keep=100, sink=4, recent=10, table=FAKE, lens=FAKE, new=FAKE, blocks=2, kc=FAKE, sc=FAKE, vc=FAKE, vsc=FAKE,
           kept=FAKE, new_lens=FAKE2, wo=FAKE2, ws=FAKE, nbytes=BIG):
    return L.dsa_grouped_evict(dims or _dims(), w, keep, sink, recent, table, lens, new, blocks, kc, sc, vc, vsc, kept, new_lens, wo, ws, nbytes,
                               None)


def test_evict_refusals(L):
    for name in ("w", "table", "lens", "new", "kc", "sc", "vc", "vsc", "kept", "new_lens", "wo"):
        assert _evict(L, **{name: None}) == 1, name
    assert _evict(L, kc=ODD) == 1 and _evict(L, vc=ODD) == 1
    assert _evict(L, keep=0) == 1 and _evict(L, keep=129) == 1 and _evict(L, sink=-1) == 1 and _evict(L, recent=-1) == 1
    assert _evict(L, sink=50, recent=51) == 1 and _evict(L, sink=(1 << 31) - 1, recent=(1 << 31) - 1) == 1
    assert _evict(L, blocks=0) == 1 and _evict(L, blocks=1 << 25) == 2
    assert _evict(L, wo=FAKE) == 1 and _evict(L, new_lens=FAKE) == 1  # in place
    assert _evict(L, ws=None) == 3 and _evict(L, ws=ODD) == 3 and _evict(L, nbytes=0) == 3
    assert _evict(L, _dims(B=1 << 20, H=1 << 10, H_kv=1 << 10, num_blocks=1), keep=128) == 2
    assert L.dsa_last_launch_count() == 0


def test_binding_refusals(L):
    """Host tensors, wrong types, shapes and sizes, and tensors that record gradients are refused in Python."""
    d = _dims()
    q, kv = torch.zeros((2, 8, 128), dtype=torch.bfloat16), torch.zeros((2, 2, 128), dtype=torch.bfloat16)
    cache, sc = torch.zeros((8, 2, 64, 128), dtype=torch.uint8), torch.zeros((8, 2))
    table, lens, ws = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1024, dtype=torch.uint8)
    w = torch.zeros((2, 2, 256))
    calls = [lambda q=q, kv=kv, w=w, c=cache: dsa.grouped_attn(d, q, c, sc, c, sc, table, lens, 0.1, weights=w, ws=ws),
             lambda q=q, kv=kv, w=w, c=cache: dsa.grouped_append(d, kv, kv, table, lens, c, sc, c, sc, ws=ws),
             lambda q=q, kv=kv, w=w, c=cache: dsa.grouped_evict(d, w, 64, table, lens, table, c, sc, c, sc, ws=ws)]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()
    grad = dict(q=q.clone().requires_grad_(), kv=kv.clone().requires_grad_(), w=w.clone().requires_grad_())
    for call, name in zip(calls, ("q", "kv", "w")):
        with pytest.raises(ValueError, match="gradient"):
            call(**{name: grad[name]})
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call(**{name: grad[name]})
    rows = lambda x, T=2, h=8, n=128, dims=d: dsa._grouped_rows(x, T, h, n, dims, "q")  # noqa: E731
    assert rows(q) == (q.data_ptr(), 1024, 128)
    for bad in (q.float(), q[:1], q[:, :4], q[..., :64], q[0]):
        with pytest.raises(ValueError, match="q must"):
            rows(bad)
    with pytest.raises(ValueError, match="dense"):
        rows(torch.zeros((2, 8, 256), dtype=torch.bfloat16)[..., ::2])
    check = lambda **kw: dsa._grouped_caches(d, **{**dict(k_cache=cache, k_scale=sc, v_cache=cache, v_scale=sc, block_table=table,  # noqa: E731
                                                          seq_lens=lens, cu=None, T=2), **kw})
    check()
    for kw, what in ((dict(k_cache=cache[:7]), "k_cache"), (dict(v_cache=cache.int()), "v_cache"), (dict(k_scale=sc[:7]), "k_scale"),
                     (dict(v_scale=sc.double()), "v_scale"), (dict(block_table=table[:1]), "block_table"), (dict(seq_lens=lens.long()), "seq_lens"),
                     (dict(cu=lens), "cu"), (dict(T=3), "one row")):
        with pytest.raises(ValueError, match=what):
            check(**kw)
    with pytest.raises(ValueError, match="new_table"):
        dsa.grouped_evict(d, w, 64, table, lens, table[:1], cache, sc, cache, sc, ws=ws)
    with pytest.raises(ValueError, match="dims"):
        dsa.grouped_workspace(_raw(H=7), 2)


def _row_tile(d, T):
    """Rows of an item: as many as the average sequence has for a key head, in powers of two."""
    rows, tile = -(-T // d.B) * (d.H // d.H_kv), 8
    while tile < rows and tile < (16 if d.type == 0 or d.d_v > 128 else 32 if d.d_qk > 128 else 64):
        tile *= 2
    return tile


def test_workspace_of_the_weights(L):
    """Room for the logits of every item that T rows in B sequences can make, and no more; never less for more rows."""
    size = lambda d, T, w=0: L.dsa_grouped_workspace_size(ctypes.byref(d), T, w)  # noqa: E731
    d = _dims(B=32, max_blocks=512, H=64, H_kv=8, num_blocks=64)
    logits = 32 * 8 * 256 * 8 * 128 * 4  # sequences, key heads, tiles, heads of a group, positions, bytes
    assert logits <= size(d, 32, 1) - size(d, 32) <= logits + 4 * 32 * 64 + 1024
    d = _dims(B=64, max_blocks=512, H=32, H_kv=32, num_blocks=64)
    assert size(d, 64, 1) - size(d, 64) <= 64 * 32 * 256 * 8 * 128 * 4 + 4 * 64 * 32 + 1024
    rng = random.Random(1)
    for _ in range(300):
        H_kv = rng.choice([1, 2, 8])
        d = _dims(type=rng.choice(["f32", "bf16"]), B=rng.choice([1, 2, 5, 40]), max_blocks=rng.choice([1, 2, 9]), H_kv=H_kv,
                  H=H_kv * rng.choice([1, 3, 5, 8, 12, 16, 64, 130]), d_qk=rng.choice([64, 192]), d_v=rng.choice([64, 192]))
        T = rng.randint(1, 4 * d.B)
        cuts = sorted(rng.randint(0, T) for _ in range(d.B - 1))
        G, tile = d.H // d.H_kv, _row_tile(d, T)
        items = sum(-(-n * G // tile) for n in (b - a for a, b in zip([0] + cuts, cuts + [T])))
        room = size(d, T, 1) - size(d, T)
        assert room >= items * tile * d.H_kv * ((d.max_blocks + 1) // 2) * 512 + 4 * T * d.H, (d.B, T, G, tile)
        for w in (0, 1):
            sizes = [size(d, n, w) for n in range(T + 1)]
            assert sizes == sorted(sizes)


def test_overlapping_outputs_are_refused(L):
    """Weights and lengths that are written while others still read them, by whatever part of them."""
    at = lambda n: ctypes.c_void_p((1 << 20) + n)  # noqa: E731
    size = 4 * 2 * 2 * 4 * 64  # bytes of the weights of 2 sequences, 2 heads and 4 blocks
    for off in (256, size - 256, -256, -size // 2 + 256):  # (the new ones have 2 blocks)
        assert _evict(L, wo=at(off)) == 1, off
    assert _evict(L, new_lens=at(4)) == 1 and _evict(L, new_lens=at(-4)) == 1
    for off in (256, size - 256, -256, 256 - size):
        assert _attn(L, w=FAKE, wo=at(off)) == 1, off
    for off in (0, size, -size):  # itself, or beside it: up to the workspace, which is too small
        assert _attn(L, w=FAKE, wo=at(off), nbytes=0) == 3, off
    assert _evict(L, wo=at(size), nbytes=0) == 3 and _evict(L, wo=at(-size // 2), nbytes=0) == 3 and _evict(L, new_lens=at(8), nbytes=0) == 3
    assert L.dsa_last_launch_count() == 0


def test_widths_of_rows():
    """What is as large as needed is taken; what is larger has whole rows in its last dimensions."""
    for shape in ((4, 6), (24,), (30,), (2, 12), (4, 2, 3), (5, 6), (2, 2, 6), (7, 2, 3), (1, 4, 3, 2)):
        dsa._row_width(torch.empty(shape), 6, 24, "x")
    for shape in ((4, 7), (2, 13), (4, 12), (5, 2, 4), (4, 2, 4)):
        with pytest.raises(ValueError, match="rows of x must have 6"):
            dsa._row_width(torch.empty(shape), 6, 24, "x")
