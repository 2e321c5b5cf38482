"""Edges of the attention block (AttentionW4A4): rows that no sequence owns or
that belong to a refused one, beside the O linear's one tensor scale; calls on
several streams and captured ones, and the workspaces of each."""
import pytest
import torch

from nvfp4_w4a4_quantized_03_b200 import inputs, mq
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu
HID, HQ, HKV, D, P = 512, 8, 2, 64, 16


def _block(seed=0, positions=5000):
    w_qkv = inputs.weight_bf16((HQ + 2 * HKV) * D, HID, seed=seed)
    w_o = inputs.weight_bf16(HID, HQ * D, seed=seed + 1)
    return mq.AttentionW4A4(w_qkv.to(dev()), w_o.to(dev()), HQ, HKV, D, mq.rope_table(positions, D, device=dev()))


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def _x(T, seed=0):
    return torch.randn(T, HID, generator=torch.Generator().manual_seed(seed)).bfloat16().to(dev())


def _steps(block, x, cache, cu, lens, table, max_q, max_len, precise=False):
    """The block's calls one by one; rows that the attention does not write are zero in the O linear's input."""
    T = x.shape[0]
    qkv = (block.qkv_precise if precise else block.qkv)(x)
    q = torch.zeros(T, HQ, D, dtype=torch.bfloat16, device=dev())
    out = torch.zeros_like(q)
    ws = mq.workspace(mq.mq_kv_attention_workspace_bytes(table.shape[0], HQ, HKV, D, max_q, max_len), dev())
    mq.mq_rope_kv_append(qkv, block.rope, cu, lens, table, *cache.tensors(), q)
    mq.mq_kv_attention(q, cu, lens, table, *cache.tensors(), out, ws, max_q, max_len, D ** -0.5)
    return (block.o_precise if precise else block.o)(out.view(T, -1))


@pytest.fixture
def poisoned(monkeypatch):
    """Memory that torch hands out uninitialised holds `value`."""
    def poison(value):
        empty, empty_like = torch.empty, torch.empty_like

        def fill(t):
            return t.fill_(value) if t.is_floating_point() and t.is_cuda else t
        monkeypatch.setattr(torch, "empty", lambda *a, **k: fill(empty(*a, **k)))
        monkeypatch.setattr(torch, "empty_like", lambda *a, **k: fill(empty_like(*a, **k)))
    return poison


@pytest.mark.parametrize("value", [float("nan"), 1e30, float("inf")])
def test_rows_of_nobody_leave_the_others_alone(poisoned, value):
    """A batch of two prompts padded to more rows: the prompts' rows are those of the unpadded call."""
    block, table = _block(), torch.arange(16, dtype=torch.int32, device=dev()).view(2, 8)
    x = _x(150)
    x[103:] = 0
    args = (_i32(0, 70, 103), _i32(70, 33), table, 70, 128)
    want = block(x[:103], mq.PagedKVCache(16, P, HKV, D, dev()), *args)
    poisoned(value)
    got = block(x, mq.PagedKVCache(16, P, HKV, D, dev()), *args)
    assert block.status() == mq.MQ_OK
    assert torch.equal(got[:103], want)
    assert (got[103:] == 0).all()


@pytest.mark.parametrize("value", [float("nan"), 1e30])
def test_a_refused_sequence_leaves_the_others_alone(poisoned, value):
    """One of three sequences is longer than max_len: reported, the others as step by step."""
    block, table = _block(1), torch.arange(48, dtype=torch.int32, device=dev()).view(3, 16)
    x = _x(120, 1)
    args = (_i32(0, 50, 80, 120), _i32(50, 200, 60), table, 50, 128)
    want = _steps(block, x, mq.PagedKVCache(48, P, HKV, D, dev()), *args)
    poisoned(value)
    got = block(x, mq.PagedKVCache(48, P, HKV, D, dev()), *args)
    assert block.status() == -1
    assert torch.equal(got, want) and torch.isfinite(got).all()


@pytest.mark.parametrize("value", [float("nan"), 1e30])
def test_a_sequence_longer_than_the_rotary_table_leaves_the_others_alone(poisoned, value):
    """The append leaves the rows of positions that the table does not have; the attention does not take up what
    memory held in their place."""
    block, table = _block(2, positions=64), torch.arange(48, dtype=torch.int32, device=dev()).view(3, 16)
    x = _x(120, 2)
    cu, lens = _i32(0, 50, 80, 120), _i32(50, 90, 60)
    want = _steps(block, x, mq.PagedKVCache(48, P, HKV, D, dev()), cu, lens, table, 50, 64)
    poisoned(value)
    got = block(x, mq.PagedKVCache(48, P, HKV, D, dev()), cu, lens, table, 50, 200)
    assert block.status() == -1
    assert torch.equal(got, want) and torch.isfinite(got).all()


def test_the_default_stream_by_its_address():
    """stream=0 is the default stream, whatever the current one: the call stands behind what it holds."""
    block, table, (old, new) = _block(3), _i32(0, 1)[None], (_x(1, 5), _x(1, 6))
    args = (_i32(0, 1), _i32(1), table, 1, 32, True)
    want = block(new, mq.PagedKVCache(2, P, HKV, D, dev()), *args)
    x, cache, side = old.clone(), mq.PagedKVCache(2, P, HKV, D, dev()), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                                        # about 10 ms on the default stream
    x.copy_(new)
    with torch.cuda.stream(side):
        got = block(x, cache, *args, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def _two(precise, seed):
    """Two batches for one block: long contexts (split keys), then what each gives alone."""
    block, T = _block(seed), 3 if precise else 90
    runs = []
    for i in range(2):
        x, cache = _x(T, 20 + i), mq.PagedKVCache(300, P, HKV, D, dev())
        for t, size in ((cache.k, 448), (cache.v, 448)):
            t.copy_((torch.randn(t.shape, generator=torch.Generator().manual_seed(i)) * 16).clamp(-size, size).to(t.dtype))
        table = torch.arange(300, dtype=torch.int32, device=dev())[None]
        runs.append((x, cache, _i32(0, T), _i32(4000 + 300 * i), table, T, 4700, precise))
    with torch.cuda.stream(torch.cuda.Stream()):
        want = [block(*r).clone() for r in runs]                          # appending the same again changes nothing
    torch.cuda.synchronize()
    return block, runs, want


@pytest.mark.parametrize("precise", [True, False])
def test_one_block_on_two_streams_at_once(precise):
    """Each call is as it is alone; the first stream is still busy when the second one's first call begins."""
    block, runs, want = _two(precise, 7)
    streams = [torch.cuda.Stream() for _ in runs]
    outs = [[], []]
    with torch.cuda.stream(streams[0]):
        torch.cuda._sleep(10_000_000)                                    # about 5 ms, the workspaces' fill behind it
    for turn in range(6):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                outs[i].append(block(*runs[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(y, want[i]) for y in outs[i]), i
    assert block.status() == mq.MQ_OK


def test_workspaces_of_streams():
    """One per stream, made anew only where a call needs more."""
    spaces, s = mq._Workspaces(keep=True), torch.cuda.Stream()
    a = spaces.get(1000, torch.device("cuda"))
    b = spaces.get(1000, dev(), s)
    c = spaces.get(1000, dev(), s.cuda_stream)
    with torch.cuda.stream(s):
        assert spaces.get(10, dev()) is b is c and spaces.last is b
    assert a is not b and spaces.get(1000, dev()) is a
    d = spaces.get(1001, dev())
    assert d is not a and d.numel() >= 1001 and spaces.replaced == [a]
    assert spaces.get(1000, dev(), s) is b and spaces.get(1000, dev(), 0) is d
    torch.cuda.synchronize()
    assert not b.any() and not d.any()
    with pytest.raises(ValueError):
        spaces.get(10, torch.device("cpu"))
    with pytest.raises(ValueError):
        spaces.get(10, dev(), "a stream")


@pytest.mark.parametrize("precise", [True, False])
def test_two_captured_calls_at_once(precise):
    """Two graphs captured one after the other on the same stream, replayed on two at once, a call on a third."""
    block, runs, want = _two(precise, 8)
    ys = [torch.empty_like(w) for w in want]
    graphs, streams = [], [torch.cuda.Stream() for _ in range(3)]
    for r, y in zip(runs, ys):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=streams[0]):
            block(*r, out=y)
            block(*r, out=y)                                             # the same workspace: one after the other
    held = {k: ws for k, ws in block._spaces.by_place.items() if k[2]}
    assert len(held) == 2 and not any(ws.any() for ws in held.values()) and block.status() == mq.MQ_OK
    third = (runs[0][0], mq.PagedKVCache(300, P, HKV, D, dev()), *runs[0][2:])
    for t, s in zip(third[1].tensors(), runs[0][1].tensors()):
        t.copy_(s)
    torch.cuda.synchronize()
    for _ in range(6):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        with torch.cuda.stream(streams[2]):
            y = block(*third)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([*ys, y], [*want, want[0]]))
    assert block.status() == mq.MQ_OK


@pytest.mark.parametrize("warm", [True, False])
@pytest.mark.parametrize("precise", [True, False])
def test_a_captured_call_outlives_larger_ones(precise, warm):
    """A graph captured at one size, with or without a call before it, then calls that need larger workspaces of every
    kind, then memory handed out anew: the replay is as before and writes nothing of others."""
    block, other, table = _block(9), _block(9), torch.arange(300, dtype=torch.int32, device=dev())[None]
    T = 2 if precise else 20
    x, cache, y = _x(T, 30), mq.PagedKVCache(300, P, HKV, D, dev()), torch.empty(T, HID, dtype=torch.bfloat16, device=dev())
    args = (_i32(0, T), _i32(1500), table, T, 1500, precise)
    want = other(x, mq.PagedKVCache(300, P, HKV, D, dev()), *args)
    if warm:
        block(x, cache, *args, out=y)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        block(x, cache, *args, out=y)
    for stream in (None, s):
        with torch.cuda.stream(stream):
            block(_x(900, 31), mq.PagedKVCache(300, P, HKV, D, dev()), _i32(0, 900), _i32(4000), table, 900, 4800)
    torch.cuda.synchronize()
    others = [torch.full((n,), 7, dtype=torch.uint8, device=dev()) for n in [1 << k for k in range(9, 22)] * 8]
    cache.k_scale.fill_(1.0), cache.v_scale.fill_(1.0)
    cache.k.view(torch.uint8).zero_(), cache.v.view(torch.uint8).zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert all((t == 7).all() for t in others)
    assert block.status() == mq.MQ_OK


def test_a_captured_linear_and_mlp_outlive_larger_calls():
    lin = mq.LinearW4A4(inputs.weight_bf16(256, HID, seed=1).to(dev()))
    mlp = mq.MLPW4A4(inputs.weight_bf16(512, HID, seed=2).to(dev()), inputs.weight_bf16(HID, 256, seed=3).to(dev()))
    x = _x(40, 40)
    want = [f(x) for f in (lin, mlp)]
    ys = [torch.empty_like(y) for y in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for f, y in zip((lin, mlp), ys):
            f(x, y)
    for f in (lin, mlp):
        f(_x(3000, 41))
    others = [torch.full((n,), 7, dtype=torch.uint8, device=dev()) for n in [1 << k for k in range(9, 22)] * 8]
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ys, want)) and all((t == 7).all() for t in others)


def test_status_of_workspaces_that_were_too_small_later():
    """What a call reported is still there after one that needed a larger workspace; once read, it is gone."""
    block, table = _block(10), torch.arange(300, dtype=torch.int32, device=dev())[None]
    assert block.status() == mq.MQ_OK                                    # before the first call
    cache = mq.PagedKVCache(300, P, HKV, D, dev())
    block(_x(1), cache, _i32(0, 1), _i32(60), table, 1, 50, True)        # longer than the call allows
    block(_x(1), cache, _i32(0, 1), _i32(4000), table, 1, 4800, True)
    assert len(block._kept) == 1
    assert block.status() == -1
    assert block.status() == mq.MQ_OK


def test_status_of_the_linears_inside():
    block, table = _block(11), _i32(0, 1)[None]
    block(_x(20), mq.PagedKVCache(2, P, HKV, D, dev()), _i32(0, 20), _i32(20), table, 20, 32)
    assert block.status() == mq.MQ_OK
    for lin in (block.qkv, block.o):
        lin._ws[8:12].view(torch.int32).fill_(mq.MQ_ERR_TIMEOUT)         # as a product whose wait ran out leaves it
        assert block.status() == mq.MQ_ERR_TIMEOUT
        assert block.status() == mq.MQ_OK


def test_tensors_of_another_device_than_the_current_one_are_refused():
    """Before anything is enqueued (the library launches on the current device)."""
    lin = mq.LinearW4A4(inputs.weight_bf16(64, 64, seed=1).to(dev()))
    with pytest.raises(ValueError, match="the current device is cuda:0"):
        lin._spaces.get(256, torch.device("cuda", torch.cuda.device_count()))
    with pytest.raises(ValueError, match="device tensor expected"):
        lin(torch.zeros(2, 64, dtype=torch.bfloat16))
