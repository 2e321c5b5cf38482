"""Edges of the attention over the paged E4M3 cache (mq_kv_attention), in the
form for few rows and in the tcgen05 form: a NaN at every place of a group of 16
keys, page numbers outside the pool, partial results joined at either head
dimension, page scales far apart.  Plain forms and bounds as in test_gpu_kv."""
import pytest
import torch

from nvfp4_w4a4_quantized_03_b200 import mq
from tests import kv_helpers as kv
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


def _attend(bt, d, q, scale, status=mq.MQ_OK):
    out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device=dev())
    ws = mq.workspace(mq.mq_kv_attention_workspace_bytes(len(bt.seqs), q.shape[1], bt.H, bt.D, bt.max_q, bt.max_len), dev())
    mq.mq_kv_attention(q.to(dev()), out=out, ws=ws, max_q=bt.max_q, max_len=bt.max_len, scale=scale, **d)
    assert mq.mq_read_status(ws) == status
    return out.cpu()


def _q(bt, heads, seed):
    return torch.randn(bt.T, heads, bt.D, generator=torch.Generator().manual_seed(seed)).bfloat16()


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("new,length,first", [(7, 57, 41), (40, 57, 34), (40, 1500, 1464), (150, 300, 225)])
def test_a_nan_at_every_place_of_a_group(new, length, first, head_dim, where):
    """Sequence i has a NaN in K or V at position first + i, through the append: the rows that see it are NaN, the
    others what the plain form gives."""
    bt = kv.Batch([(length, length)] * 16, 16, 1, head_dim, seed=new)
    g = torch.Generator().manual_seed(length)
    qkv = torch.randn(bt.T, 4 * head_dim, generator=g).bfloat16()
    for i in range(16):
        at = (3 if where == "v" else 2) * head_dim + int(torch.randint(head_dim, (1,), generator=g))
        qkv[int(bt.cu[i]) + first + i, at] = float("nan")
    d = bt.to(dev())
    mq.mq_rope_kv_append(qkv.to(dev()), None, q_out=torch.empty(bt.T, 2, head_dim, dtype=torch.bfloat16, device=dev()), **d)
    # the last `new` tokens of every sequence attend
    last = kv.Batch([(new, length)] * 16, 16, 1, head_dim)
    last.table, last.pages = bt.table, bt.pages
    last.k, last.v = (d[n].view(torch.uint8).cpu() for n in ("k_codes", "v_codes"))
    last.ks, last.vs = d["k_scales"].cpu(), d["v_scales"].cpu()
    q = _q(last, 2, 5)
    got = _attend(last, last.to(dev()), q, 0.125).view(16, new, 2, head_dim)
    sees = torch.arange(length - new, length)[None, :] >= first + torch.arange(16)[:, None]
    assert torch.isnan(got[sees]).all()
    want, bound = (t.view(16, new, 2, head_dim) for t in kv.attention_plain(last, q, 0.125))
    kv.close_to(got[~sees], want[~sees], bound[~sees])


@pytest.mark.parametrize("number", ["behind", "negative"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("new,length", [(1, 70), (4, 70), (30, 70), (30, 2100)])
def test_keys_of_a_page_outside_the_pool_are_left_out(new, length, head_dim, number):
    """As if the sequence did not hold them; a sequence without any valid page sees nothing.  The status word says so."""
    bad, page = 1, 16
    bt = kv.Batch([(new, length), (new, length), (new, length)], page, 2, head_dim, seed=length, extra_pages=3).fill()
    # the pool's first page is nobody's, NaN all over
    bt.table[bt.table >= 0] += 1
    bt.pages += 1
    bt.k, bt.v = (torch.cat([torch.full_like(t[:1], 0x7F), t]) for t in (bt.k, bt.v))
    bt.ks, bt.vs = (torch.cat([t[:1], t]) for t in (bt.ks, bt.vs))
    q = _q(bt, 8, 1)
    # the same without the page: all rows stand behind it
    short = kv.Batch([(new, length - page)] * 3, page, 2, head_dim, extra_pages=0)
    short.table = torch.cat([bt.table[:, :bad], bt.table[:, bad + 1:]], 1)
    short.pages, short.k, short.v, short.ks, short.vs = bt.pages, bt.k, bt.v, bt.ks, bt.vs
    want, bound = kv.attention_plain(bt, q, 0.125)
    want[:new], bound[:new] = (t[:new] for t in kv.attention_plain(short, q, 0.125))
    want[new:2 * new] = bound[new:2 * new] = 0
    d = bt.to(dev())
    d["page_table"][0, bad] = d["page_table"][1, :] = bt.pages if number == "behind" else -2
    got = _attend(bt, d, q, 0.125, status=-1)
    assert (got[new:2 * new] == 0).all()
    kv.close_to(got, want, bound)


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("seqs,group", [([(20, 3000)], 1), ([(33, 2500)], 2), ([(60, 4000), (3, 1100), (25, 30)], 1),
                                        ([(65, 2049)], 4), ([(300, 5000)], 2), ([(1, 9000)], 4), ([(2, 20000), (1, 17)], 8)])
def test_joined_chunks(seqs, group, head_dim):
    """Keys split over blocks and joined, up to 64 rows per cell (a warp per row) and more (a thread per row)."""
    bt = kv.Batch(seqs, 16, 2, head_dim, seed=len(seqs) + group).fill()
    q = _q(bt, 2 * group, group)
    got = _attend(bt, bt.to(dev()), q, bt.D ** -0.5)
    kv.close_to(got, *kv.attention_plain(bt, q, bt.D ** -0.5))


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("new", [1, 40])
def test_pages_of_zeros_beside_large_ones(new, head_dim):
    """V all zero (the least scale there is, 2^-96) beside V up to 448 2^12: the zeros keep their share of the softmax."""
    bt = kv.Batch([(new, 96)], 16, 1, head_dim, seed=3).fill()
    for i in (1, 3):
        p = int(bt.table[0, i])
        bt.v[p], bt.vs[p] = 0, 2.0 ** -96
    p = int(bt.table[0, 0])
    bt.vs[p] *= 2.0 ** 12 / float(bt.vs[p])
    q = _q(bt, 2, 4)
    got = _attend(bt, bt.to(dev()), q, 0.125)
    kv.close_to(got, *kv.attention_plain(bt, q, 0.125))
