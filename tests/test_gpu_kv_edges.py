"""Edges of the attention over the paged E4M3 cache (mq_kv_attention), in the
form for few rows and in the tcgen05 form: a NaN at every place of a group of 16
keys.  Plain forms and bounds as in test_gpu_kv."""
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
