"""Refusals of the rotary, read-back and prompt entry points, before anything is launched (no GPU needed), and the
frequencies, which are computed on the host."""
import ctypes
import math

import pytest
import torch

import indexer_top_sparse_paged_gb300 as dsa
from indexer_top_sparse_paged_gb300.build import build_library

FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: every call below fails its checks first
ODD = ctypes.c_void_p((1 << 20) + 4)
BIG = 1 << 30


@pytest.fixture(scope="module")
def L():
    build_library()
    return dsa.lib()


def test_frequency_refusals_and_values(L):
    f = (ctypes.c_double * 32)()
    ok = (64, 10000.0, 2, 40.0, 4096.0, 32.0, 1.0, f)
    assert L.dsa_rope_frequencies(*ok) == 0
    assert f[0] == 1.0 and abs(f[31] * 40 / 10000 ** (-62 / 64) - 1) < 1e-12
    for i, bad, st in ((0, 63, 1), (0, 0, 1), (0, 514, 2), (1, 0.0, 1), (1, 1.0, 1), (1, math.inf, 1), (2, 3, 2), (2, -1, 2), (3, 0.5, 1),
                       (3, math.nan, 1), (4, 0.0, 1), (5, 0.5, 1), (6, 0.0, 1), (7, None, 1)):
        a = list(ok)
        a[i] = bad
        assert L.dsa_rope_frequencies(*a) == st, (i, bad)


def _rope(L, x=None, type_=1, n=1, rot=64, freq=FAKE, lens=None, pos=FAKE, T=4, scale=1.0):
    x = x or dsa.RopeTensor(1 << 20, 1 << 21, 8, 0, 512, 64, 512, 64)
    arr = (dsa.RopeTensor * 4)(x, x, x, x)
    return L.dsa_rope(type_, arr, n, rot, freq, lens, pos, T, scale, 0, None)


def test_rope_refusals(L):
    R = dsa.RopeTensor
    assert _rope(L, T=0) == 0 and L.dsa_last_launch_count() == 0
    assert _rope(L, type_=2) == 2 and _rope(L, n=5) == 2 and _rope(L, rot=514) == 2
    assert _rope(L, n=0) == 1 and _rope(L, rot=7) == 1 and _rope(L, T=-1) == 1 and _rope(L, scale=math.inf) == 1
    assert _rope(L, freq=None) == 1 and _rope(L, freq=ODD) == 1 and _rope(L, pos=None) == 1
    assert _rope(L, R(None, 1 << 21, 8, 0, 512, 64, 512, 64)) == 1 and _rope(L, R(1 << 20, None, 8, 0, 512, 64, 512, 64)) == 1
    assert _rope(L, R((1 << 20) + 1, 1 << 21, 8, 0, 512, 64, 512, 64)) == 1  # not on an element
    assert _rope(L, R(1 << 20, 1 << 21, 8, 2, 512, 64, 512, 64)) == 1        # no such layout
    assert _rope(L, R(1 << 20, 1 << 21, -1, 0, 512, 64, 512, 64)) == 1
    assert _rope(L, R(1 << 20, 1 << 20, 8, 0, 512, 64, 1024, 64)) == 1       # in place through other strides


def _dims(**kw):
    d = dict(mode="mxfp8", B=2, max_blocks=4, num_blocks=8, H_I=64, d_I=128, H=128, d=576, d_v=512, K=256, kv="fp8")
    d.update(kw)
    return dsa.make_dims(**d)


def test_append_rope_refusals(L):
    def call(dims=None, r=(64, 0, 1, 512, 0, 1.0), freq=FAKE, k=FAKE, scale=FAKE, seq=None, T=2, ws=FAKE, nbytes=BIG):
        return L.dsa_cache_append_rope(ctypes.byref(dims or _dims()), ctypes.byref(dsa.RopeAppend(*r)) if r else None, freq, k, FAKE,
                                       FAKE, FAKE, seq, None, T, FAKE, scale, FAKE, ws, nbytes, None)
    assert call(_dims(B=1), T=0, seq=FAKE) == 0 and L.dsa_last_launch_count() == 0
    assert call(r=None) == 1 and call(freq=None) == 1 and call(freq=ODD) == 1 and call(k=None) == 1 and call(k=ODD) == 1
    for r, st in (((63, 0, 1, 512, 0, 1.0), 1), ((258, 0, 1, 0, 0, 1.0), 2), ((64, 65, 1, 512, 0, 1.0), 1), ((64, 0, 1, 513, 0, 1.0), 1),
                  ((64, -2, 1, 512, 0, 1.0), 1), ((64, 0, 2, 512, 0, 1.0), 1), ((64, 0, 1, 512, 0, math.nan), 1), ((130, 0, 1, 0, 0, 1.0), 1)):
        assert call(r=r) == st, r
    assert call(scale=None) == 1 and call(T=3) == 1 and call(T=-1, seq=FAKE) == 1
    assert call(ws=None) == 3 and call(ws=ODD) == 3 and call(nbytes=100) == 3
    assert call(_dims(d_I=48), r=(32, 0, 1, 512, 0, 1.0)) == 2 and call(_dims(d=584)) == 2


def test_cache_read_refusals(L):
    def call(dims=None, kc=FAKE, sc=FAKE, kv=FAKE, table=FAKE, cu=FAKE, R=5, ko=FAKE, vo=FAKE, ws=FAKE, nbytes=BIG):
        return L.dsa_cache_read(ctypes.byref(dims or _dims()), kc, sc, kv, table, FAKE, None, cu, R, ko, vo, ws, nbytes, None)
    assert call(R=0) == 0 and L.dsa_last_launch_count() == 0
    assert call(R=-1) == 1 and call(ko=None, vo=None) == 1 and call(table=None) == 1 and call(cu=None) == 1
    assert call(kc=None) == 1 and call(sc=None) == 1 and call(kv=None) == 1 and call(ko=ODD) == 1 and call(vo=ODD) == 1
    assert call(ws=None) == 3 and call(nbytes=0) == 3
    assert call(_dims(d_I=48)) == 2 and call(_dims(mode="bf16_kfp8", d_I=24)) == 2 and call(_dims(d=584)) == 2
    assert L.dsa_cache_read(None, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, 1, FAKE, FAKE, FAKE, BIG, None) == 1


def _prompt(**kw):
    p = dict(type=1, B=2, H=8, H_kv=2, d_qk=128, d_v=128, causal=1, q_stride_t=1024, q_stride_h=128, k_stride_t=256, k_stride_h=128,
             v_stride_t=256, v_stride_h=128)
    p.update(kw)
    return dsa.PromptDims(*p.values())


def test_prompt_refusals(L):
    size = lambda d, T=100: L.dsa_prompt_workspace_size(ctypes.byref(d), T)  # noqa: E731
    assert size(_prompt()) > 0 and L.dsa_prompt_workspace_size(None, 4) == 0 and size(_prompt(), -1) == 0

    def call(dims=None, q=FAKE, k=FAKE, v=FAKE, cu_q=FAKE, cu_k=FAKE, Tq=100, Tk=100, scale=0.1, out=FAKE, ws=FAKE, nbytes=BIG):
        return L.dsa_prompt_attn(ctypes.byref(dims or _prompt()), q, k, v, cu_q, cu_k, Tq, Tk, scale, out, None, ws, nbytes, None)
    assert call(Tq=0) == 0 and L.dsa_last_launch_count() == 0
    for kw, st in ((dict(type=2), 2), (dict(B=0), 1), (dict(H=7), 1), (dict(H=0), 1), (dict(H_kv=0), 1), (dict(d_qk=264), 2), (dict(d_v=264), 2),
                   (dict(d_qk=100), 2), (dict(d_v=12), 2), (dict(q_stride_t=1023), 1), (dict(k_stride_h=-128), 1), (dict(v_stride_t=1 << 40), 1)):
        assert size(_prompt(**kw)) == 0 and call(_prompt(**kw)) == st, kw
    assert call(q=None) == 1 and call(k=None) == 1 and call(v=None) == 1 and call(cu_q=None) == 1 and call(cu_k=None) == 1
    assert call(q=ODD) == 1 and call(k=ODD) == 1 and call(v=ODD) == 1 and call(out=ODD) == 1 and call(out=None) == 1
    assert call(Tq=-1) == 1 and call(Tk=-1) == 1 and call(Tq=1 << 30) == 2
    for s in (0.0, -1.0, math.nan, math.inf):
        assert call(scale=s) == 1
    assert call(ws=None) == 3 and call(ws=ODD) == 3 and call(nbytes=size(_prompt()) - 1) == 3


def test_binding_refusals(L):
    """Host tensors, wrong types and shapes are refused in Python."""
    x, freq = torch.zeros((4, 2, 64)), torch.ones(32, dtype=torch.float64)
    pos = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.rope(x, freq, q_pos=pos)
    with pytest.raises(ValueError, match="same number"):
        dsa.rope([x, x], freq, q_pos=pos, layout=["half"])
    with pytest.raises(ValueError, match="scaling"):
        dsa.rope_frequencies(64, scaling="none", device="cpu")
    with pytest.raises(dsa.DsaError):
        dsa.rope_frequencies(7, device="cpu")
    q, k = torch.zeros((4, 8, 64)), torch.zeros((4, 2, 64))
    with pytest.raises(ValueError, match="same tokens"):
        dsa.prompt_dims(q, k, k[:3], 1)
    with pytest.raises(ValueError, match="all float32"):
        dsa.prompt_dims(q, k.bfloat16(), k, 1)
    with pytest.raises(ValueError, match="dense"):
        dsa.prompt_dims(q.transpose(1, 2), k, k, 1)
    d = dsa.prompt_dims(q, k, k, 1)
    with pytest.raises(ValueError, match="differ"):
        dsa.prompt_attn(d, q[:, ::2], k, k, pos, pos, 0.1, ws=x)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.prompt_attn(d, q, k, k, pos, pos, 0.1, ws=x)
    assert L.dsa_last_launch_count() == 0


def test_tensors_that_record_gradients_are_refused(L):
    """None of these calls records anything for autograd; a gradient that would get lost is an error, and under
    no_grad the same tensors go on to the next check."""
    x, freq, i32 = torch.zeros((4, 2, 64), requires_grad=True), torch.ones(32, dtype=torch.float64), torch.zeros(8, dtype=torch.int32)
    q, k = torch.zeros((4, 8, 64)), torch.zeros((4, 2, 64))
    ws, row = torch.zeros(1024, dtype=torch.uint8), torch.zeros((1, 576), dtype=torch.bfloat16)
    dims = _dims(B=1)
    new = torch.zeros((1, 128), dtype=torch.bfloat16, requires_grad=True)
    calls = [lambda: dsa.rope(x, freq, q_pos=i32[:4]), lambda: dsa.rope([q, x * 1], freq, q_pos=i32[:4]),
             lambda: dsa.rope(x.detach(), freq, q_pos=i32[:4], out=x),
             lambda: dsa.cache_append_rope(dims, freq, new, row, i32, i32, ws, ws, ws, ws=ws),
             lambda: dsa.cache_read(dims, ws, ws, new, i32, i32, i32, 1, ws=ws)]
    for a, b, c in ((q.clone().requires_grad_(), k, k), (q, k.clone().requires_grad_(), k), (q, k, k.clone().requires_grad_())):
        calls.append(lambda a=a, b=b, c=c: dsa.prompt_attn(dsa.prompt_dims(a, b, c, 1), a, b, c, i32, i32, 0.1, ws=ws))
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call()
    assert L.dsa_last_launch_count() == 0


def test_prompts_longer_than_32_bits_count_are_refused(L):
    """The keys of a call are counted in 32 bits and rounded up to tiles: a count that leaves no room for that is
    refused (it gave rows without keys), whatever the strides that make so many keys cheap."""
    for type_, strides in ((0, (0, 8, 0, 8)), (1, (0, 8, 0, 8)), (1, (8, 8, 8, 8))):
        dims = _prompt(type=type_, B=1, H=1, H_kv=1, d_qk=8, d_v=8, q_stride_t=8, q_stride_h=8, k_stride_t=strides[0], k_stride_h=strides[1],
                       v_stride_t=strides[2], v_stride_h=strides[3])
        for Tk in ((1 << 31) - 1, (1 << 31) - (1 << 16)):
            assert L.dsa_prompt_attn(ctypes.byref(dims), FAKE, FAKE, FAKE, FAKE, FAKE, 1, Tk, 0.1, FAKE, None, None, BIG, None) == 2
        # the largest count goes on to the next check
        assert L.dsa_prompt_attn(ctypes.byref(dims), FAKE, FAKE, FAKE, FAKE, FAKE, 1, (1 << 31) - (1 << 16) - 1, 0.1, FAKE, None, None, BIG,
                                 None) == 3


def test_frequencies_outside_of_64_bits_are_refused(L):
    """A stretched base or a frequency that overflows is no set of frequencies (all but the first came out as 0, or
    the last ones as infinite); the outermost bases that do not overflow give what the definition gives."""
    f = (ctypes.c_double * 32)()
    for base, scaling, factor in ((1e300, 1, 1e10), (1e-300, 1, 1.7e308), (5e-324, 0, 1.0), (1e-310, 0, 1.0)):
        assert L.dsa_rope_frequencies(64, base, scaling, factor, 4096.0, 32.0, 1.0, f) == 1 or all(math.isfinite(x) and x > 0 for x in f), base
    assert L.dsa_rope_frequencies(64, 1e300, 1, 1e10, 4096.0, 32.0, 1.0, f) == 1
    assert L.dsa_rope_frequencies(64, 5e-324, 0, 1.0, 4096.0, 32.0, 1.0, f) == 1
    for base in (1e300, 1e-300):
        assert L.dsa_rope_frequencies(64, base, 0, 1.0, 4096.0, 32.0, 1.0, f) == 0
        assert all(abs(f[i] / base ** (-2.0 * i / 64) - 1) < 1e-12 for i in range(32))
