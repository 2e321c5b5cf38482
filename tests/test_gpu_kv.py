"""The rotary append to the paged E4M3 cache and the attention over it
(mq_rope_kv_append, mq_kv_attention) against plain CPU forms: the append bit
for bit (every step of it is one binary32 operation) and its rotation against
64 bits, the attention element by element within the bound that
kv_helpers.attention_plain derives."""
import math

import pytest
import torch

from nvfp4_w4a4_quantized_03_b200 import mq
from tests import kv_helpers as kv
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


def _append(bt, qkv, table, q_heads, rot_dim, interleaved, row_stride=None):
    d = bt.to(dev())
    q = torch.full((bt.T, q_heads, bt.D), -7.0, dtype=torch.bfloat16, device=dev())
    x = qkv.to(dev())
    if row_stride:
        wide = torch.full((bt.T, row_stride), float("nan"), dtype=torch.bfloat16, device=dev())
        wide[:, :x.shape[1]] = x
        x = wide[:, :x.shape[1]]
    ws = mq.workspace(mq.mq_workspace_bytes(), dev())
    mq.mq_rope_kv_append(x, None if table is None else table.to(dev()), q_out=q, ws=ws, rot_dim=rot_dim,
                         interleaved=interleaved, **d)
    torch.cuda.synchronize()
    return d, q.cpu(), mq.mq_read_status(ws)


def _check_append(bt, qkv, table, q_heads, rot_dim, interleaved, row_stride=None):
    d, q, status = _append(bt, qkv, table, q_heads, rot_dim, interleaved, row_stride)
    assert status == mq.MQ_OK
    want64 = None
    if rot_dim:
        # |fl(fl(ac) - fl(bs)) - (ac - bs)| <= 2 u (|ac| + |bs|) (1 + u), u = 2^-24; |c|, |s| <= 1 + u
        x = qkv.double().view(bt.T, -1, bt.D)[:, :q_heads]
        size = x.abs().amax(2, keepdim=True)
    ref = kv.append_plain(bt, qkv, table, q_heads, rot_dim, interleaved, torch.float32)
    mine = ~torch.isnan(ref)
    assert torch.equal(q[mine], ref.bfloat16()[mine])
    assert (q[~mine] == -7.0).all()                                  # rows that are nobody's stay
    for name, want in (("k_codes", bt.k), ("v_codes", bt.v)):
        assert torch.equal(d[name].view(torch.uint8).cpu(), want), name
    assert torch.equal(d["k_scales"].cpu(), bt.ks) and torch.equal(d["v_scales"].cpu(), bt.vs)
    if rot_dim:
        want64 = kv.append_plain(bt, qkv, table, q_heads, rot_dim, interleaved, torch.float64)
        bound = (6 * 2.0 ** -24 * size).expand_as(want64)
        kv.close_to(q[mine], want64[mine], bound[mine])


def _qkv(bt, q_heads, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(bt.T, q_heads + 2 * bt.H, bt.D, generator=g) * size
    x *= torch.exp(torch.randn(q_heads + 2 * bt.H, bt.D, generator=g))
    return x.bfloat16().view(bt.T, -1)


SEQS = {
    "one token": [(1, 1)],
    "one token later": [(1, 38)],
    "decode": [(1, 16), (1, 17), (1, 33), (0, 40), (1, 1), (1, 129)],
    "chunks": [(70, 70), (3, 131), (0, 0), (129, 200), (1, 128), (17, 18)],
    "left padding": [(5, 3), (40, 0), (2, 2)],
}


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("seqs", list(SEQS))
def test_append(seqs, head_dim, page):
    i = list(SEQS).index(seqs)
    rot_dim, interleaved = [(head_dim, False), (head_dim // 2, True), (16, False), (head_dim, True), (0, False)][i]
    bt = kv.Batch(SEQS[seqs], page, 2, head_dim, seed=i, extra_rows=3).fill()
    table = kv.rope(256, rot_dim) if rot_dim else None
    _check_append(bt, _qkv(bt, 6, i + 50), table, 6, rot_dim, interleaved)


@pytest.mark.parametrize("q_heads,kv_heads,rot_dim,interleaved", [(1, 1, 128, False), (32, 8, 128, False),
                                                                  (7, 7, 32, True), (20, 4, 96, False),
                                                                  (24, 8, 96, True)])
def test_append_heads_and_layouts(q_heads, kv_heads, rot_dim, interleaved):
    bt = kv.Batch([(37, 90), (1, 64)], 64, kv_heads, 128, seed=3, extra_rows=1).fill()
    width = (q_heads + 2 * kv_heads) * 128
    _check_append(bt, _qkv(bt, q_heads, 9), kv.rope(90, rot_dim), q_heads, rot_dim, interleaved, row_stride=width + 24)


def test_append_many_rows():
    """Blocks of several rows of Q (2048 rows and more), a sequence border inside one."""
    bt = kv.Batch([(1001, 1001), (0, 5), (1100, 1111)], 128, 1, 64, seed=4, extra_rows=2)
    _check_append(bt, _qkv(bt, 2, 10), kv.rope(1200, 64), 2, 64, False)


def test_append_one_by_one_equals_the_plain_form_at_every_step():
    """A page's scale grows as larger tokens come; the earlier codes follow."""
    bt = kv.Batch([(1, 20)], 16, 1, 64, seed=5)
    table = kv.rope(64, 64)
    for step in range(20):
        bt.seqs[0] = (1, step + 1)
        bt.lens[0] = step + 1
        _check_append(bt, _qkv(bt, 2, 100 + step, size=2.0 ** (step % 7 - 3)), table, 2, 64, False)


@pytest.mark.parametrize("size", [0.0, 1e-37, 3e38, 2.0 ** 119, 448.0, 449.0])
def test_append_extreme_sizes(size):
    bt = kv.Batch([(3, 5), (2, 2)], 16, 1, 64, seed=6).fill()
    x = torch.randn(bt.T, 3 * 64, generator=torch.Generator().manual_seed(1)).clamp(-1, 1) * size
    x[0, 64], x[1, 128] = size, -size
    _check_append(bt, x.bfloat16(), None, 1, 0, False)


def test_append_nan_reaches_only_the_rows_that_see_it():
    bt = kv.Batch([(40, 40)], 16, 1, 64, seed=7)
    qkv = _qkv(bt, 1, 3)
    qkv[20, 128 + 5] = float("nan")                                  # V of token 20
    qkv[30, 64 + 9] = float("nan")                                   # K of token 30
    d, q, status = _append(bt, qkv, None, 1, 0, False)
    assert status == mq.MQ_OK
    out = _attend(bt, d, q.to(dev()), 0.125)
    assert torch.isfinite(out[:20]).all() and torch.isnan(out[20:]).all()


def test_append_tables_that_do_not_cover_the_batch():
    """Positions beyond the rotary table, page numbers outside the pool: reported, nothing written."""
    bt = kv.Batch([(3, 20), (4, 4)], 16, 1, 64, seed=8).fill()
    before = bt.k.clone(), bt.ks.clone()
    bt.table[0, 1] = bt.pages                                        # the page of positions 16..19
    d, q, status = _append(bt, _qkv(bt, 1, 4), kv.rope(20, 64), 1, 64, False)
    assert status == -1
    own = int(bt.table[1, 0])
    got = d["k_codes"].view(torch.uint8).cpu()
    others = [p for p in range(bt.pages) if p != own]
    assert torch.equal(got[others], before[0][others]) and torch.equal(d["k_scales"].cpu()[others], before[1][others])
    bt.table[0, 1] = 0 if own else 1
    _, q, status = _append(bt, _qkv(bt, 1, 4), kv.rope(19, 64), 1, 64, False)   # position 19 has no row
    assert status == -1 and (q[2] == -7.0).all() and (q[0] != -7.0).any()


# -- attention --------------------------------------------------------------------

def _attend(bt, d, q, scale, max_q=None, max_len=None, ws=None):
    out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device=dev())
    max_q, max_len = max_q or bt.max_q, bt.max_len if max_len is None else max_len
    if ws is None:
        need = mq.mq_kv_attention_workspace_bytes(len(bt.seqs), q.shape[1], bt.H, bt.D, max_q, max_len)
        ws = mq.workspace(need, dev())
    mq.mq_kv_attention(q, out=out, ws=ws, max_q=max_q, max_len=max_len, scale=scale, **d)
    torch.cuda.synchronize()
    assert mq.mq_read_status(ws) == mq.MQ_OK
    return out.cpu()


def _check_attention(bt, q_heads, scale=None, q_size=1.0, seed=0, **kw):
    q = (torch.randn(bt.T, q_heads, bt.D, generator=torch.Generator().manual_seed(seed)) * q_size).bfloat16()
    scale = bt.D ** -0.5 if scale is None else scale
    got = _attend(bt, bt.to(dev()), q.to(dev()), scale, **kw)
    want, bound = kv.attention_plain(bt, q, scale)
    nobody = torch.isnan(want)
    assert (got[nobody] == -7.0).all()
    print("worst error / bound:", kv.close_to(got[~nobody], want[~nobody], bound[~nobody]))


ATTEND = {
    "one key": [(1, 1)],
    "decode": [(1, 15), (1, 16), (1, 17), (0, 9), (1, 700), (1, 1), (1, 129)],
    "few": [(3, 3), (2, 130), (4, 64), (0, 0), (1, 31)],
    "chunks": [(70, 70), (33, 333), (129, 129), (1, 257)],
    "left padding": [(5, 3), (7, 0), (2, 40)],
}


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("seqs", list(ATTEND))
def test_attention(seqs, head_dim, page):
    i = list(ATTEND).index(seqs)
    bt = kv.Batch(ATTEND[seqs], page, 2, head_dim, seed=20 + i, extra_rows=2).fill()
    _check_attention(bt, 2 * [4, 1, 3, 2, 5][i], seed=i)


@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 9, 16, 17, 33, 128])
@pytest.mark.parametrize("new", [1, 2, 5])
def test_attention_groups(group, new):
    bt = kv.Batch([(new, 77), (new, 5)], 32, 1, 64, seed=group).fill()
    _check_attention(bt, group, seed=new)


@pytest.mark.parametrize("length", [1, 63, 64, 65, 1023, 4097, 9001])
@pytest.mark.parametrize("new", [1, 4, 40])
def test_attention_lengths(length, new):
    """One sequence, split over the device in chunks that the last block joins."""
    bt = kv.Batch([(min(new, length), length)], 16, 1, 128, seed=length).fill()
    _check_attention(bt, 4, seed=length)


@pytest.mark.parametrize("new", [1, 50])
def test_attention_pages_of_very_different_sizes(new):
    bt = kv.Batch([(new, 400)], 16, 1, 64, seed=31).fill(spread=20)
    _check_attention(bt, 4, seed=1)


@pytest.mark.parametrize("new", [1, 50])
@pytest.mark.parametrize("q_size,k_size,v_size", [(30.0, 1.0, 1.0), (1e-30, 1.0, 1e-20), (1e30, 1e-30, 1e20),
                                                  (1.0, 0.0, 1.0), (1.0, 1.0, 0.0)])
def test_attention_sizes(new, q_size, k_size, v_size):
    """Sharp softmax (one key takes all), flat softmax, operands far from one."""
    bt = kv.Batch([(new, 300)], 32, 1, 128, seed=32).fill(k_size, v_size)
    _check_attention(bt, 2, q_size=q_size, seed=2)


@pytest.mark.parametrize("new", [1, 40])
def test_attention_strided_q_larger_bounds_and_a_workspace_used_before(new):
    """q as a slice of the QKV product; max_q and max_len larger than the batch needs; the workspace of a call of
    other sizes."""
    bt = kv.Batch([(new, 90), (1, 3000)], 64, 2, 128, seed=33).fill()
    other = kv.Batch([(1, 9000)], 64, 1, 128, seed=34).fill()
    ws = mq.workspace(64 << 20, dev())
    qkv = torch.randn(bt.T, (8 + 4) * 128, generator=torch.Generator().manual_seed(5)).bfloat16()
    want, bound = kv.attention_plain(bt, qkv[:, :1024].reshape(bt.T, 8, 128), 0.05)
    for _ in range(2):
        q = qkv.to(dev())[:, :1024].unflatten(1, (8, 128))
        got = _attend(bt, bt.to(dev()), q, 0.05, max_q=100, max_len=5000, ws=ws)
        kv.close_to(got, want, bound)
        _check_attention(other, 4, ws=ws)


def test_attention_lengths_beyond_the_call_are_reported():
    bt = kv.Batch([(1, 40), (2, 50), (1, 20)], 16, 1, 64, seed=35).fill()
    q = torch.randn(bt.T, 2, 64).bfloat16()
    want, bound = kv.attention_plain(bt, q, 0.125)
    for max_q, max_len, table, bad in ((1, 50, None, [1, 2]), (2, 45, None, [1, 2]), (2, 50, 3, [1, 2])):
        d = bt.to(dev())
        if table:
            d["page_table"] = d["page_table"][:, :table].contiguous()           # 48 positions
        out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device=dev())
        ws = mq.workspace(mq.mq_kv_attention_workspace_bytes(3, 2, 1, 64, max_q, max_len), dev())
        mq.mq_kv_attention(q.to(dev()), out=out, ws=ws, max_q=max_q, max_len=max_len, scale=0.125, **d)
        assert mq.mq_read_status(ws) == -1
        out = out.cpu()
        assert (out[bad] == -7.0).all()
        good = [r for r in range(bt.T) if r not in bad]
        kv.close_to(out[good], want[good], bound[good])


# Batches of more tiles than run at once: their blocks take the sequences in the order of the keys they see.
WAVES = {
    "ragged": [(600, 900), (37, 2000), (0, 50), (1, 1), (599, 599), (130, 1200), (33, 2), (600, 601)],
    "alike": [(300, 300)] * 8,
    "more than a warp": [(3 + 11 * i % 40, 5 + 37 * i % 300) for i in range(40)],
    "as many as are ordered": [(i % 7, (17 * i) % 90) for i in range(127)] + [(40, 90)],
    "more than are ordered": [(i % 4, (17 * i) % 90) for i in range(130)],
}


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("seqs", list(WAVES))
def test_attention_more_tiles_than_run_at_once(seqs, head_dim):
    bt = kv.Batch(WAVES[seqs], 16, 2, head_dim, seed=40, extra_rows=2).fill()
    _check_attention(bt, 16, seed=3, max_q=max(600, bt.max_q))


def test_attention_more_tiles_than_run_at_once_lengths_beyond_the_call():
    """Sequences that the call refuses among others: reported, left alone, the others computed."""
    bt = kv.Batch([(600, 700), (20, 1000), (70, 80), (5, 2000), (601, 601), (1, 700)], 16, 2, 64, seed=41).fill()
    q = torch.randn(bt.T, 16, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    want, bound = kv.attention_plain(bt, q, 0.125)
    ws = mq.workspace(mq.mq_kv_attention_workspace_bytes(6, 16, 2, 64, 600, 1000), dev())
    out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device=dev())
    mq.mq_kv_attention(q.to(dev()), out=out, ws=ws, max_q=600, max_len=1000, scale=0.125, **bt.to(dev()))
    assert mq.mq_read_status(ws) == -1
    bad = torch.zeros(bt.T, dtype=torch.bool)
    bad[690:695] = bad[695:1296] = True                                   # the fourth (length) and the fifth (rows)
    out = out.cpu()
    assert (out[bad] == -7.0).all()
    kv.close_to(out[~bad], want[~bad], bound[~bad])


@pytest.mark.parametrize("new", [1, 40])
def test_attention_page_numbers_outside_the_pool_are_reported(new):
    bt = kv.Batch([(new, 60), (new, 60)], 16, 1, 64, seed=36).fill()
    q = torch.randn(bt.T, 2, 64).bfloat16()
    want, bound = kv.attention_plain(bt, q, 0.125)
    d = bt.to(dev())
    d["page_table"][0, 1] = bt.pages
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev())
    ws = mq.workspace(mq.mq_kv_attention_workspace_bytes(2, 2, 1, 64, new, 60), dev())
    mq.mq_kv_attention(q.to(dev()), out=out, ws=ws, max_q=new, max_len=60, scale=0.125, **d)
    assert mq.mq_read_status(ws) == -1
    kv.close_to(out.cpu()[new:], want[new:], bound[new:])


def test_attention_repeats_exactly():
    bt = kv.Batch([(1, 5000), (3, 200)], 64, 2, 128, seed=37).fill()
    q = torch.randn(bt.T, 8, 128).bfloat16().to(dev())
    d = bt.to(dev())
    first = _attend(bt, d, q, 0.1)
    for _ in range(5):
        assert torch.equal(_attend(bt, d, q, 0.1), first)
