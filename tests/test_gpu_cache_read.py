"""dsa_cache_read: every storage mode read back bit for bit (code * scale in fp32, one rounding to bf16), ranges
inside sequences, ragged and empty batches, rows around the ranges left alone, bad entries as zeros."""
import numpy as np
import pytest
import torch

import indexer_top_sparse_paged_gb300 as dsa
import workloads as W
from cases import small_spec

pytestmark = pytest.mark.gpu

SHAPES = {"f32": dict(H_I=8, d_I=36, H=4, d=68, d_v=48), "bf16": {}, "bf16_kfp8": {}, "mxfp8": {}}
MODES = [("f32", "act"), ("bf16", "act"), ("bf16", "fp8"), ("bf16_kfp8", "act"), ("mxfp8", "fp8")]


def _dev(a):
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).cuda().view(torch.bfloat16)
    return torch.from_numpy(a).cuda()


class Cache:
    def __init__(self, mode, kv, lens, seed=500, **kw):
        kw = {**SHAPES[mode], **kw}
        c = self.case = W.generate(small_spec(mode, lens, 64, kv=kv, **kw), seed=seed)
        s = self.spec = c.spec
        self.dims = dsa.make_dims(s.mode, s.B, c.max_blocks, c.num_blocks, s.H_I, s.d_I, s.H, s.d, s.d_v, s.K, kv=s.kv)
        self.k, self.kv = _dev(c.k_I), _dev(c.kv)
        self.scale = None if c.k_I_scale is None else _dev(c.k_I_scale)
        self.table, self.lens = _dev(c.block_table), _dev(c.seq_lens)
        self.ws = dsa.workspace(self.dims, 1)

    def want(self, b, p0, n):
        s = self.spec
        pos = torch.arange(p0, p0 + n, device="cuda")
        blk = self.table[b, pos // 64].long()
        row = blk * 64 + pos % 64
        k = self.k.view(-1, s.d_I)[row]
        if s.mode == "bf16_kfp8":
            k = (k.view(torch.float8_e4m3fn).float() * self.scale[blk][:, None]).bfloat16()
        elif s.mode == "mxfp8":
            f = torch.exp2(self.scale.view(-1, s.d_I // 32)[row].float() - 127).repeat_interleave(32, 1)
            k = (k.view(torch.float8_e4m3fn).float() * f).bfloat16()
        if s.kv == "fp8":
            r = self.kv.view(-1, dsa.kv_record_bytes(s.d))[row]
            f = r[:, s.d:s.d + 4 * ((s.d + 127) // 128)].contiguous().view(torch.float32).repeat_interleave(128, 1)[:, :s.d]
            kv = (r[:, :s.d].contiguous().view(torch.float8_e4m3fn).float() * f).bfloat16()
        else:
            kv = self.kv.view(-1, s.d)[row]
        return k, kv

    def read(self, cu, R, start=None, **kw):
        i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return dsa.cache_read(self.dims, self.k, self.scale, self.kv, self.table, self.lens, i32(cu), R, i32(start),
                              ws=self.ws, **kw)


@pytest.mark.parametrize("mode,kv", MODES)
@pytest.mark.parametrize("lens,start,n", [([1], None, [1]), ([65], [64], [1]), ([200, 64, 1, 0, 333], None, [200, 64, 1, 0, 333]),
                                          ([500, 130, 70], [63, 129, 0], [300, 1, 0]), ([40] * 33, None, [40] * 33)])
def test_ranges_read_back_exactly(mode, kv, lens, start, n):
    c = Cache(mode, kv, lens)
    cu = np.concatenate(([0], np.cumsum(n))).tolist()
    k, v = c.read(cu, cu[-1], start)
    assert dsa.last_launch_count() == 1 and dsa.read_error(c.ws) == 0
    for b, m in enumerate(n):
        wk, wv = c.want(b, 0 if start is None else start[b], m)
        assert torch.equal(k[cu[b]:cu[b + 1]], wk) and torch.equal(v[cu[b]:cu[b + 1]], wv), b


@pytest.mark.parametrize("mode,kv,d,d_I", [("bf16", "fp8", 144, 64), ("mxfp8", "fp8", 576, 128), ("bf16_kfp8", "act", 576, 128), ("bf16", "act", 8, 8)])
def test_odd_widths_one_output_and_rows_left_alone(mode, kv, d, d_I):
    c = Cache(mode, kv, [100, 30, 7], d=d, d_v=min(d, 8), d_I=d_I, H=2, H_I=2)
    s = c.spec
    R = 150
    k_out = torch.full((R, s.d_I), 7.0, dtype=torch.bfloat16, device="cuda")
    kv_out = torch.full((R, s.d), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = [2, 102, 132, 139]  # two rows in front and eleven behind belong to nobody
    c.read(cu, R, k_out=k_out, kv_out=kv_out)
    assert dsa.read_error(c.ws) == 0
    for out, which in ((k_out, 0), (kv_out, 1)):
        assert bool((out[:2] == 7).all()) and bool((out[139:] == 7).all())
        for b, n in enumerate((100, 30, 7)):
            assert torch.equal(out[cu[b]:cu[b + 1]], c.want(b, 0, n)[which])
    k, none = c.read(cu, R, want_kv=False)
    assert none is None and torch.equal(k[2:139], k_out[2:139])
    none, v = c.read(cu, R, want_k=False)
    assert none is None and torch.equal(v[2:139], kv_out[2:139])
    c.read([0, 0, 0, 0], 0, k_out=k_out, kv_out=kv_out)
    assert dsa.last_launch_count() == 0


def test_positions_and_blocks_out_of_range_read_as_zeros():
    c = Cache("mxfp8", "fp8", [100, 130, 50])
    k, v = c.read([0, 110, 120, 130], 130, [0, -3, 45])
    assert dsa.read_error(c.ws) == 2
    for out, which in ((k, 0), (v, 1)):
        assert torch.equal(out[:100], c.want(0, 0, 100)[which]) and not out[100:110].any()
        assert not out[110:113].any() and torch.equal(out[113:120], c.want(1, 0, 7)[which])
        assert torch.equal(out[120:125], c.want(2, 45, 5)[which]) and not out[125:].any()
    c.table[1, 1] = c.case.num_blocks
    k, v = c.read([0, 0, 130, 130], 130)
    assert dsa.read_error(c.ws) == 1
    assert torch.equal(k[:64], c.want(1, 0, 64)[0]) and not k[64:128].any() and not v[64:128].any()
    c.table[1, 1] = 0
    assert torch.equal(k[128:], c.want(1, 128, 2)[0])


def test_append_then_read_is_the_identity_of_stored_values():
    """A row appended in rotated form comes back as rope's output rounded to its record's step: half a step is
    2^-4 of the value, 2^-10 of the tile's scale below the normal codes; bf16's own half step is 2^-8."""
    c = Cache("mxfp8", "fp8", [300, 77])
    s, rot = c.spec, 32
    freq = dsa.rope_frequencies(rot)
    n = [100, 77]
    q_seq = torch.tensor([0] * 100 + [1] * 77, dtype=torch.int32, device="cuda")
    q_pos = torch.cat((torch.arange(200, 300), torch.arange(77))).to(torch.int32).cuda()
    k_new, kv_new = torch.randn((177, s.d_I), device="cuda").bfloat16(), torch.randn((177, s.d), device="cuda").bfloat16()
    dsa.cache_append_rope(c.dims, freq, k_new, kv_new, c.table, c.lens, c.k, c.scale, c.kv, q_seq, q_pos, ws=c.ws)
    k, v = c.read([0, n[0], sum(n)], sum(n), [200, 0])
    assert dsa.read_error(c.ws) == 0
    wk, wv = k_new.float(), kv_new.float()
    dsa.rope(wk[:, None, :rot], freq, q_pos=q_pos, layout="half")
    dsa.rope(wv[:, None, s.d - rot:], freq, q_pos=q_pos)
    for got, want, group in ((k, wk, 32), (v, wv, 128)):
        pad = torch.nn.functional.pad(want, (0, -want.shape[1] % group)).view(len(want), -1, group)
        top = pad.abs().amax(-1).repeat_interleave(group, 1)[:, :want.shape[1]]
        # MX scales can leave the group's largest value above 448 steps, where it saturates: 64 of 512
        bound = want.abs() * (2.0 ** -4 + 2.0 ** -7) + top * (2.0 ** -10 / 224)
        if group == 32:
            bound = torch.maximum(bound, torch.where(want.abs() >= top * 0.875, want.abs() * 0.125 * 1.05, bound))
        assert bool(((got.float() - want).abs() <= bound).all())


def test_rows_up_to_what_32_bits_count():
    """The last rows of an output of 2^31 - 1 rows (32 GB of them, three of which are written)."""
    c = Cache("bf16", "act", [100], d=8, d_v=8, d_I=8, H=2, H_I=2)
    R = (1 << 31) - 1
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("32 GB of outputs do not fit")
    k_out = torch.empty((R, 8), dtype=torch.bfloat16, device="cuda")
    k_out[-4:] = 7
    k, _ = c.read([R - 3, R], R, [50], k_out=k_out, want_kv=False)
    assert dsa.read_error(c.ws) == 0
    assert bool((k_out[-4] == 7).all()) and torch.equal(k_out[-3:], c.want(0, 50, 3)[0])
    del k, k_out
    torch.cuda.empty_cache()
