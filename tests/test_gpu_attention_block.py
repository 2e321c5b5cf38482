"""The operators of the attention block together, as a layer uses them: QKV
linear, rotary append, attention, O linear (AttentionW4A4), prompt first and
then token by token; in captured graphs, on other streams, on caches and rows
whose offsets pass 32 bits, inside the prefill sequence; and the debug build
over the same calls."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from nvfp4_w4a4_quantized_03_b200 import inputs, mq
from nvfp4_w4a4_quantized_03_b200.sequence import PrefillSequence
from tests import kv_helpers as kv
from tests.gpu_helpers import bits, dev

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HID, HQ, HKV, D, P = 512, 8, 2, 64, 16


def _block(seed=0):
    w_qkv = inputs.weight_bf16((HQ + 2 * HKV) * D, HID, seed=seed)
    w_o = inputs.weight_bf16(HID, HQ * D, seed=seed + 1)
    return mq.AttentionW4A4(w_qkv.to(dev()), w_o.to(dev()), HQ, HKV, D, mq.rope_table(300, D, device=dev()))


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def test_prompt_then_tokens():
    """A prompt through the quantizing linears, then 20 tokens through the precise ones, two sequences: after every
    step the attention inside agrees with the plain form on what the cache then holds, and the block's output with
    its O linear on the attention's."""
    block, table = _block(), torch.tensor([[3, 0, 5, 9], [7, 2, 8, 1]], dtype=torch.int32, device=dev())
    cache = mq.PagedKVCache(10, P, HKV, D, dev())
    lens = [37, 18]
    g = torch.Generator().manual_seed(0)
    new = list(lens)
    for step in range(21):
        T = sum(new)
        x = torch.randn(T, HID, generator=g).bfloat16().to(dev())
        cu = _i32(0, new[0], T)
        y = block(x, cache, cu, _i32(*lens), table, max_q=max(new), max_len=64, precise=step > 0)
        assert block.status() == mq.MQ_OK
        # the same steps one by one, on the cache as it now is (appending the same tokens changes nothing)
        qkv = (block.qkv_precise if step else block.qkv)(x)
        q = torch.empty(T, HQ, D, dtype=torch.bfloat16, device=dev())
        before = [t.clone() for t in cache.tensors()]
        mq.mq_rope_kv_append(qkv, block.rope, cu, _i32(*lens), table, *cache.tensors(), q)
        for a, b in zip(before, cache.tensors()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        bt = kv.Batch([(n, length) for n, length in zip(new, lens)], P, HKV, D)
        bt.table, bt.pages = table.cpu(), 10
        bt.k, bt.v = (t.view(torch.uint8).cpu() for t in cache.tensors()[:2])
        bt.ks, bt.vs = (t.cpu() for t in cache.tensors()[2:])
        want, bound = kv.attention_plain(bt, q.cpu(), D ** -0.5)
        out = torch.empty_like(q)
        mq.mq_kv_attention(q, cu, _i32(*lens), table, *cache.tensors(), out, block._ws, max(new), 64, D ** -0.5)
        kv.close_to(out.cpu(), want, bound)
        assert torch.equal(y, (block.o_precise if step else block.o)(out.view(T, -1)))
        new = [1, 1]
        lens = [n + 1 for n in lens]


def test_decode_step_in_a_graph():
    """A captured step replayed with other tokens, lengths and pages in the same tensors."""
    block = _block(2)
    pages = torch.arange(64, dtype=torch.int32, device=dev()).view(4, 16)
    g = torch.Generator().manual_seed(1)
    x, lens, cu = torch.zeros(4, HID, dtype=torch.bfloat16, device=dev()), _i32(1, 1, 1, 1), _i32(0, 1, 2, 3, 4)
    caches = [mq.PagedKVCache(64, P, HKV, D, dev()) for _ in range(2)]
    y = torch.empty(4, HID, dtype=torch.bfloat16, device=dev())
    block(x, caches[0], cu, lens, pages, 1, 200, precise=True, out=y)      # workspaces, launch attributes
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        block(x, caches[0], cu, lens, pages, 1, 200, precise=True, out=y)
    caches[0].k.view(torch.uint8).zero_(), caches[0].v.view(torch.uint8).zero_()
    for step in range(40):
        x.copy_(torch.randn(4, HID, generator=g).bfloat16())
        lens.copy_(_i32(step + 1, step // 2 + 1, 1, 5 * (step % 3) + 1))
        graph.replay()
        want = block(x, caches[1], cu, lens, pages, 1, 200, precise=True)
        assert torch.equal(y, want)
    assert block.status() == mq.MQ_OK


def test_two_streams_with_their_own_workspaces():
    """Two batches at once on two streams, workspace and cache apart: each as it is alone."""
    runs = []
    for i in range(2):
        bt = kv.Batch([(1, 4000 + i), (3, 500)], 64, 2, 128, seed=50 + i).fill()
        d, q = bt.to(dev()), torch.randn(bt.T, 8, 128, generator=torch.Generator().manual_seed(i)).bfloat16().to(dev())
        need = mq.mq_kv_attention_workspace_bytes(2, 8, 2, 128, 3, 4100)
        runs.append((d, q, torch.empty_like(q), mq.workspace(need, dev()), torch.cuda.Stream()))
    alone = []
    for d, q, out, ws, _ in runs:
        mq.mq_kv_attention(q, out=out, ws=ws, max_q=3, max_len=4100, scale=0.1, **d)
        alone.append(out.clone())
        out.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(10):
        for d, q, out, ws, s in runs:
            mq.mq_kv_attention(q, out=out, ws=ws, max_q=3, max_len=4100, scale=0.1, stream=s, **d)
    torch.cuda.synchronize()
    for (_, _, out, _, _), want in zip(runs, alone):
        assert torch.equal(out, want)


def test_sequences_that_share_pages():
    """The same full pages in two sequences' tables (a shared prefix), each appending to a page of its own."""
    bt = kv.Batch([(2, 40), (1, 37)], 16, 2, 64, seed=60, extra_pages=4).fill()
    bt.table[1, :2] = bt.table[0, :2]
    qkv = torch.randn(bt.T, (4 + 4) * 64, generator=torch.Generator().manual_seed(3)).bfloat16()
    d = bt.to(dev())
    q = torch.empty(bt.T, 4, 64, dtype=torch.bfloat16, device=dev())
    mq.mq_rope_kv_append(qkv.to(dev()), None, q_out=q, **d)
    ref = kv.append_plain(bt, qkv, None, 4, 0, False, torch.float32)
    assert torch.equal(q.cpu(), ref.bfloat16()) and torch.equal(d["k_codes"].view(torch.uint8).cpu(), bt.k)
    out = torch.empty_like(q)
    ws = mq.workspace(mq.mq_kv_attention_workspace_bytes(2, 4, 2, 64, 2, 40), dev())
    mq.mq_kv_attention(q, out=out, ws=ws, max_q=2, max_len=40, scale=0.125, **d)
    kv.close_to(out.cpu(), *kv.attention_plain(bt, q.cpu(), 0.125))


@pytest.mark.parametrize("new", [1, 40])
def test_a_cache_beyond_32_bit_offsets(new):
    """Pages at the far end of a pool of more than 2^32 bytes."""
    page, H, dim = 128, 8, 128
    pages = 2 ** 32 // (page * H * dim) + 70
    bt = kv.Batch([(new, 300)], page, H, dim, seed=70, extra_pages=0).fill()
    n = bt.pages
    d = bt.to(dev())
    big = {}
    for name in ("k_codes", "v_codes"):
        big[name] = torch.empty(pages, H, page, dim, dtype=torch.uint8, device=dev())
        big[name][pages - n:] = d[name].view(torch.uint8)
    for name in ("k_scales", "v_scales"):
        big[name] = torch.empty(pages, H, device=dev())
        big[name][pages - n:] = d[name]
    table = d["page_table"] + (pages - n)
    q = torch.randn(bt.T, 16, dim, generator=torch.Generator().manual_seed(4)).bfloat16()
    out = torch.empty(bt.T, 16, dim, dtype=torch.bfloat16, device=dev())
    ws = mq.workspace(mq.mq_kv_attention_workspace_bytes(1, 16, H, dim, new, 300), dev())
    args = (d["cu_rows"], d["lens"], table, *(big[k] for k in ("k_codes", "v_codes", "k_scales", "v_scales")))
    mq.mq_kv_attention(q.to(dev()), *args, out, ws, new, 300, 0.1)
    kv.close_to(out.cpu(), *kv.attention_plain(bt, q, 0.1))
    # the append to the same pages
    qkv = torch.randn(bt.T, (16 + 2 * H) * dim, generator=torch.Generator().manual_seed(5)).bfloat16()
    q_out = torch.empty_like(out)
    mq.mq_rope_kv_append(qkv.to(dev()), None, *args, q_out, rot_dim=0)
    kv.append_plain(bt, qkv, None, 16, 0, False, torch.float32)
    assert torch.equal(big["k_codes"][pages - n:].cpu(), bt.k) and torch.equal(big["v_codes"][pages - n:].cpu(), bt.v)
    assert torch.equal(big["k_scales"][pages - n:].cpu(), bt.ks)


def test_rows_beyond_32_bit_offsets():
    """Rows of the QKV product 2^27 elements apart."""
    bt = kv.Batch([(20, 33)], 16, 1, 64, seed=80).fill()
    qkv = torch.randn(20, 4 * 64, generator=torch.Generator().manual_seed(6)).bfloat16()
    wide = torch.empty(20 * 2 ** 27, dtype=torch.bfloat16, device=dev()).view(20, 2 ** 27)
    x = wide[:, :4 * 64]
    x.copy_(qkv)
    d = bt.to(dev())
    q = torch.empty(20, 2, 64, dtype=torch.bfloat16, device=dev())
    table = kv.rope(40, 64)
    mq.mq_rope_kv_append(x, table.to(dev()), q_out=q, **d)
    ref = kv.append_plain(bt, qkv, table, 2, 64, False, torch.float32)
    assert torch.equal(q.cpu(), ref.bfloat16()) and torch.equal(d["v_codes"].view(torch.uint8).cpu(), bt.v)
    out = torch.empty_like(q)
    ws = mq.workspace(mq.mq_kv_attention_workspace_bytes(1, 2, 1, 64, 20, 33), dev())
    mq.mq_kv_attention(x[:, :128].unflatten(1, (2, 64)), out=out, ws=ws, max_q=20, max_len=33, scale=0.125, **d)
    kv.close_to(out.cpu(), *kv.attention_plain(bt, qkv[:, :128].reshape(20, 2, 64), 0.125))


def test_the_binding_s_refusals_on_the_device():
    bt = kv.Batch([(2, 5)], 16, 1, 64).fill()
    d = bt.to(dev())
    x = torch.zeros(2, 3 * 64, dtype=torch.bfloat16, device=dev())
    q = torch.zeros(2, 1, 64, dtype=torch.bfloat16, device=dev())
    ws = mq.workspace(1 << 20, dev())
    ok = dict(out=torch.empty_like(q), ws=ws, max_q=2, max_len=5, scale=0.1)
    for bad in (dict(k_codes=d["k_codes"].float()), dict(v_codes=d["v_codes"][:1]), dict(k_scales=d["k_scales"].double()),
                dict(lens=d["lens"].long()), dict(page_table=d["page_table"][:, :0].repeat(2, 1)), dict(cu_rows=d["cu_rows"][:1]),
                dict(lens=d["lens"].cpu()), dict(k_codes=d["k_codes"].transpose(2, 3))):
        with pytest.raises(ValueError):
            mq.mq_kv_attention(q, **{**d, **bad}, **ok)
        with pytest.raises(ValueError):
            mq.mq_rope_kv_append(x, None, **{**d, **bad}, q_out=q)
    with pytest.raises(ValueError):
        mq.mq_kv_attention(q.float(), **d, **ok)
    with pytest.raises(ValueError):
        mq.mq_kv_attention(q.transpose(0, 1), **d, **ok)
    with pytest.raises(ValueError):
        mq.mq_rope_kv_append(x[:, :64], None, q_out=q, **d)
    with pytest.raises(ValueError):
        mq.mq_rope_kv_append(x, torch.zeros(9, 64, device=dev()), q_out=q, rot_dim=32, **d)
    with pytest.raises(mq.MQError) as e:
        mq.mq_kv_attention(q, **d, **{**ok, "ws": ws[:256]})
    assert e.value.status == -5
    with pytest.raises(mq.MQError):
        mq.mq_kv_attention(q, **d, **{**ok, "scale": 0.0})
    with pytest.raises(ValueError):
        mq.mq_linear_w4a16(x, ws, ws, ws, 64, q)
    with pytest.raises(ValueError):
        mq.mq_linear_w4a16(x, ws[:10], ws, torch.ones(1, device=dev()), 64, q)


def test_prefill_sequence_with_attention():
    """Eager and replayed runs agree; the last layer's attention agrees with the plain form on sampled rows."""
    seq = PrefillSequence(layers=2, tokens=500, device=dev(), attention=True)
    seq.run()
    torch.cuda.synchronize()
    assert seq.status() == mq.MQ_OK
    eager = [bits(y) for y in seq.y] + [bits(seq.x[seq.i_o])]
    seq.capture()
    for y in seq.y:
        y.fill_(float("nan"))
    seq.replay()
    seq.replay()
    torch.cuda.synchronize()
    assert seq.status() == mq.MQ_OK
    for e, y in zip(eager, seq.y + [seq.x[seq.i_o]]):
        assert np.array_equal(bits(y), e)
    cache = seq.caches[-1]
    bt = kv.Batch([(500, 500)], 64, 8, 128, extra_pages=0)
    bt.table = seq.batch[2].cpu()
    bt.k, bt.v = cache.k.view(torch.uint8).cpu(), cache.v.view(torch.uint8).cpu()
    bt.ks, bt.vs = cache.k_scale.cpu(), cache.v_scale.cpu()
    want, bound = kv.attention_plain(bt, seq.q.cpu(), 128 ** -0.5)
    kv.close_to(seq.x[seq.i_o].view(500, 32, 128).cpu(), want, bound)


# -- the bounds-check build ---------------------------------------------------------------

def _workloads():
    out = []
    for i, (seqs, page, heads, group, dim) in enumerate([([(1, 5), (1, 300), (0, 7)], 16, 2, 4, 128), ([(70, 200), (3, 3)], 32, 1, 7, 64),
                                                         ([(300, 300)], 128, 2, 2, 128), ([(1, 9000)], 64, 1, 8, 64),
                                                         ([(9, 2)], 64, 1, 1, 64)]):
        bt = kv.Batch(seqs, page, heads, dim, seed=90 + i, extra_rows=1).fill()
        d = bt.to("cuda")
        Hq = heads * group
        x = torch.randn(bt.T, (Hq + 2 * heads) * dim, generator=torch.Generator().manual_seed(i)).bfloat16().cuda()
        q = torch.zeros(bt.T, Hq, dim, dtype=torch.bfloat16, device="cuda")
        mq.mq_rope_kv_append(x, mq.rope_table(9000, dim), q_out=q, interleaved=bool(i % 2), **d)
        y = torch.zeros_like(q)
        ws = mq.workspace(mq.mq_kv_attention_workspace_bytes(len(seqs), Hq, heads, dim, bt.max_q, bt.max_len), "cuda")
        mq.mq_kv_attention(q, out=y, ws=ws, max_q=bt.max_q, max_len=bt.max_len, scale=0.1, **d)
        out += [bits(q), bits(y)] + [d[k].view(torch.uint8).cpu().numpy() for k in ("k_codes", "v_codes", "k_scales", "v_scales")]
    for M, N, K in [(1, 64, 64), (5, 300, 320), (16, 1000, 1024), (33, 130, 4096), (64, 256, 192)]:
        lin = mq.LinearW4A16(inputs.weight_bf16(N, K, seed=N, device="cuda"))
        out.append(bits(lin(inputs.activation_bf16(M, K, seed=M, outlier_channels=2, device="cuda"))))
    torch.cuda.synchronize()
    return out


def test_debug_build_checks_pass_and_match_the_release_build(tmp_path):
    assert not mq.mq_is_debug_build()
    release = _workloads()
    out = tmp_path / "dbg.npz"
    code = ("import sys, numpy as np; sys.path.insert(0, %r); "
            "from nvfp4_w4a4_quantized_03_b200 import mq; assert mq.mq_is_debug_build(); "
            "from tests.test_gpu_attention_block import _workloads; r = _workloads(); "
            "np.savez(%r, hits=np.array([mq.mq_debug_bounds_hits()]), *r)") % (ROOT, str(out))
    p = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, MQ_DEBUG="1"), cwd=ROOT, capture_output=True,
                       text=True, timeout=600)
    assert p.returncode == 0, p.stderr[-3000:]
    got = np.load(out)
    assert int(got["hits"][0]) == 0
    for i, r in enumerate(release):
        assert np.array_equal(got[f"arr_{i}"], r), i


# -- few rows (a slot per row), odd lengths -----------------------------------------------

@pytest.mark.parametrize("seqs", [[(2, 17)], [(2, 1)], [(3, 2), (1, 1)], [(2, 0)], [(1, 16), (2, 33), (0, 3)], [(4, 18), (1, 32)]])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("q_heads,kv_heads", [(3, 3), (8, 1)])
def test_a_few_rows(seqs, page, q_heads, kv_heads):
    """Rows that cross a page, rows of padding in front, next to one another: the append bit for bit, the attention
    of its Q over what it stored."""
    bt = kv.Batch(seqs, page, kv_heads, 64, seed=len(seqs), extra_rows=1).fill()
    table = kv.rope(64, 32)
    qkv = torch.randn(bt.T, (q_heads + 2 * kv_heads) * 64, generator=torch.Generator().manual_seed(7)).bfloat16()
    d = bt.to(dev())
    q = torch.full((bt.T, q_heads, 64), -7.0, dtype=torch.bfloat16, device=dev())
    ws = mq.workspace(mq.mq_kv_attention_workspace_bytes(len(seqs), q_heads, kv_heads, 64, bt.max_q, bt.max_len), dev())
    mq.mq_rope_kv_append(qkv.to(dev()), table.to(dev()), q_out=q, ws=ws, interleaved=True, **d)
    ref = kv.append_plain(bt, qkv, table, q_heads, 32, True, torch.float32)
    mine = ~torch.isnan(ref)
    assert torch.equal(q.cpu()[mine], ref.bfloat16()[mine]) and (q.cpu()[~mine] == -7.0).all()
    assert torch.equal(d["k_codes"].view(torch.uint8).cpu(), bt.k) and torch.equal(d["v_codes"].view(torch.uint8).cpu(), bt.v)
    assert torch.equal(d["k_scales"].cpu(), bt.ks)
    out = torch.full_like(q, -7.0)
    mq.mq_kv_attention(q, out=out, ws=ws, max_q=bt.max_q, max_len=bt.max_len, scale=0.125, **d)
    assert mq.mq_read_status(ws) == mq.MQ_OK
    want, bound = kv.attention_plain(bt, q.cpu(), 0.125)
    nobody = torch.isnan(want)
    assert (out.cpu()[nobody] == -7.0).all()
    kv.close_to(out.cpu()[~nobody], want[~nobody], bound[~nobody])


@pytest.mark.parametrize("new", [1, 30])
def test_lengths_below_zero(new):
    """A length below zero is one of zero: nothing is appended, the rows see nothing."""
    bt = kv.Batch([(new, 5), (new, 40)], 16, 1, 64, seed=9).fill()
    d = bt.to(dev())
    d["lens"][0] = -2 ** 31
    before = d["k_codes"].view(torch.uint8).clone()
    qkv = torch.randn(bt.T, 4 * 64, generator=torch.Generator().manual_seed(8)).bfloat16().to(dev())
    q = torch.zeros(bt.T, 2, 64, dtype=torch.bfloat16, device=dev())
    mq.mq_rope_kv_append(qkv, None, q_out=q, **d)
    own = bt.table[1, :3].long()
    others = [p for p in range(bt.pages) if p not in own.tolist()]
    assert torch.equal(d["k_codes"].view(torch.uint8)[others], before[others])
    out = torch.full_like(q, -7.0)
    ws = mq.workspace(mq.mq_kv_attention_workspace_bytes(2, 2, 1, 64, new, 40), dev())
    mq.mq_kv_attention(q, out=out, ws=ws, max_q=new, max_len=40, scale=0.125, **d)
    assert mq.mq_read_status(ws) == mq.MQ_OK
    assert (out[:new] == 0).all() and (out[new:] != -7.0).any()


def test_a_workspace_that_grows_keeps_the_old_one():
    block = _block(5)
    a = block.workspace(1, 1, 100, dev())
    b = block.workspace(8, 1, 100000, dev())
    assert b.numel() > a.numel() and any(w is a for w in block._kept)


@pytest.mark.parametrize("as_address", [False, True])
def test_block_on_another_stream_than_the_current_one(as_address):
    """The block's intermediate tensors are that stream's: what the current stream allocates meanwhile is elsewhere."""
    block = _block(6)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(4, HID, generator=g).bfloat16().to(dev())
    table = torch.arange(4, dtype=torch.int32, device=dev())[:, None].contiguous()
    lens, cu = _i32(1, 1, 1, 1), _i32(0, 1, 2, 3, 4)
    caches = [mq.PagedKVCache(4, P, HKV, D, dev()) for _ in range(2)]
    want = block(x, caches[0], cu, lens, table, 1, P, precise=True)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)                                    # about 10 ms: the calls below stand behind it
    got = block(x, caches[1], cu, lens, table, 1, P, precise=True, stream=s.cuda_stream if as_address else s)
    sizes = [(4, (HQ + 2 * HKV) * D), (4, HQ, D), (4, HQ, D), (4, HID)]
    others = [torch.full(size, 7.0, dtype=torch.bfloat16, device=dev()) for size in sizes * 4]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all((t == 7.0).all() for t in others)
