"""Host checks of the cache, attention and bf16-activation linear calls: what
include/mq.h refuses is refused before any device call, by the C entry points
and by the binding; the rotary table and the tests' own plain forms hold."""
import ctypes
import math

import pytest
import torch

from nvfp4_w4a4_quantized_03_b200 import build, mq
from tests import kv_helpers as kv

P16 = ctypes.c_void_p(4096)              # an aligned dummy address; never dereferenced


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_scales", "v_scales")] + [
        ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Seqs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("cu_rows", "lens", "page_table")] + [
        ("max_pages", ctypes.c_int64), ("batch", ctypes.c_int32), ("reserved", ctypes.c_int32)]


@pytest.fixture(scope="module")
def L():
    build.build()
    return mq.lib()


def _cache(**kw):
    return Cache(**{**dict(k_codes=4096, v_codes=4096, k_scales=4096, v_scales=4096, num_pages=8, page_size=64,
                           kv_heads=8, head_dim=128, reserved=0), **kw})


def _seqs(**kw):
    return Seqs(**{**dict(cu_rows=4096, lens=4096, page_table=4096, max_pages=4, batch=2, reserved=0), **kw})


def _append(L, cache=None, seqs=None, **kw):
    a = {**dict(qkv=P16, T=3, stride=48 * 128, q_heads=32, rope=P16, max_pos=100, rot=128, il=0, q=P16, ws=None, n=0), **kw}
    return L.mq_rope_kv_append(a["qkv"], a["T"], a["stride"], a["q_heads"], a["rope"], a["max_pos"], a["rot"], a["il"],
                               None if cache == 0 else ctypes.byref(cache or _cache()),
                               None if seqs == 0 else ctypes.byref(seqs or _seqs()), a["q"], a["ws"], a["n"], None)


def _attend(L, cache=None, seqs=None, **kw):
    a = {**dict(q=P16, T=3, stride=32 * 128, q_heads=32, max_q=2, max_len=100, scale=0.1, out=P16, ws=P16, n=1 << 30), **kw}
    return L.mq_kv_attention(a["q"], a["T"], a["stride"], a["q_heads"], ctypes.byref(cache or _cache()),
                             ctypes.byref(seqs or _seqs()), a["max_q"], a["max_len"], a["scale"], a["out"], a["ws"],
                             a["n"], None)


INVALID, SHAPE, ALIGN, WORKSPACE = -1, -2, -3, -5
BAD_CACHE = [(INVALID, dict(k_codes=0)), (INVALID, dict(v_scales=0)), (INVALID, dict(reserved=1)),
             (SHAPE, dict(page_size=48)), (SHAPE, dict(page_size=256)), (SHAPE, dict(head_dim=96)),
             (SHAPE, dict(kv_heads=0)), (SHAPE, dict(num_pages=0)), (SHAPE, dict(kv_heads=7)),
             (ALIGN, dict(k_codes=4104)), (ALIGN, dict(k_scales=4097))]
BAD_SEQS = [(INVALID, dict(cu_rows=0)), (INVALID, dict(page_table=0)), (SHAPE, dict(batch=0)),
            (SHAPE, dict(max_pages=0)), (SHAPE, dict(max_pages=1 << 40)), (ALIGN, dict(lens=4098))]


@pytest.mark.parametrize("want,kw", BAD_CACHE)
def test_caches_that_are_refused(L, want, kw):
    assert _append(L, cache=_cache(**kw)) == want
    assert _attend(L, cache=_cache(**kw)) == want


@pytest.mark.parametrize("want,kw", BAD_SEQS)
def test_batches_that_are_refused(L, want, kw):
    assert _append(L, seqs=_seqs(**kw)) == want
    assert _attend(L, seqs=_seqs(**kw)) == want


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(qkv=None)), (INVALID, dict(q=None)), (INVALID, dict(il=2)), (INVALID, dict(rope=None)),
    (INVALID, dict(max_pos=0)), (SHAPE, dict(T=0)), (SHAPE, dict(T=(1 << 24) + 1)), (SHAPE, dict(rot=24)),
    (SHAPE, dict(rot=144)), (SHAPE, dict(rot=-16)), (SHAPE, dict(stride=48 * 128 - 8)), (SHAPE, dict(stride=48 * 128 + 4)),
    (SHAPE, dict(q_heads=33)), (SHAPE, dict(q_heads=0)), (ALIGN, dict(qkv=ctypes.c_void_p(4100))),
    (ALIGN, dict(rope=ctypes.c_void_p(4100))), (WORKSPACE, dict(ws=P16, n=128)),
    (ALIGN, dict(ws=ctypes.c_void_p(4100), n=256))])
def test_appends_that_are_refused(L, want, kw):
    assert _append(L, **kw) == want


def test_append_without_tables(L):
    assert _append(L, cache=0) == INVALID and _append(L, seqs=0) == INVALID


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(q=None)), (INVALID, dict(out=None)), (INVALID, dict(scale=0.0)), (INVALID, dict(scale=-1.0)),
    (INVALID, dict(scale=float("nan"))), (INVALID, dict(scale=float("inf"))), (SHAPE, dict(max_q=0)),
    (SHAPE, dict(max_len=-1)), (SHAPE, dict(max_len=1 << 31)), (SHAPE, dict(max_q=1 << 25)),
    (SHAPE, dict(stride=32 * 128 - 8)), (SHAPE, dict(q_heads=8 * 129)), (WORKSPACE, dict(ws=None)),
    (WORKSPACE, dict(n=256)), (ALIGN, dict(ws=ctypes.c_void_p(4096 + 16))), (ALIGN, dict(q=ctypes.c_void_p(4100)))])
def test_attentions_that_are_refused(L, want, kw):
    assert _attend(L, **kw) == want


def test_attention_workspace(L):
    f = mq.mq_kv_attention_workspace_bytes
    one = f(1, 32, 8, 128, 1, 100)                      # one chunk: the header and the tickets
    assert one == f(64, 32, 8, 128, 1, 8) and one % 256 == 0
    assert f(1, 32, 8, 128, 1, 100000) > one            # partial results
    assert f(1, 33, 8, 128, 1, 100) == 0 and f(0, 32, 8, 128, 1, 100) == 0 and f(1, 32, 8, 96, 1, 100) == 0
    # grows at most with the cells, however long the context
    assert f(1, 8, 8, 128, 1, 1 << 30) <= one + 8 * 128 * 8 * 130 * 4


def test_attention_workspace_of_more_blocks_than_a_launch_has(L):
    """batch x row tiles x kv heads of 2^31 is refused, and has no workspace size."""
    f = mq.mq_kv_attention_workspace_bytes
    assert f(1 << 20, 1024, 1024, 128, 16, 8) > 0                   # one row tile of 16: 2^30 blocks
    assert f(1 << 20, 1024, 1024, 128, 257, 8) == 0                 # two of 256


@pytest.mark.parametrize("want,M,N,K,kw", [
    (SHAPE, 0, 64, 64, {}), (SHAPE, 65, 64, 64, {}), (SHAPE, 1, 64, 96, {}), (SHAPE, 1, 0, 64, {}),
    (INVALID, 1, 64, 64, dict(x=None)), (INVALID, 1, 64, 64, dict(alpha=None)), (ALIGN, 1, 64, 64, dict(x=ctypes.c_void_p(4104))),
    (ALIGN, 1, 64, 64, dict(alpha=ctypes.c_void_p(4097)))])
def test_linears_that_are_refused(L, want, M, N, K, kw):
    a = {**dict(x=P16, alpha=P16), **kw}
    assert L.mq_linear_w4a16(a["x"], M, K, P16, P16, a["alpha"], N, P16, None) == want


def test_the_binding_refuses_what_is_not_on_the_device(L):
    """CPU tensors, wrong types and shapes are a ValueError, not an address for the library."""
    bt = kv.Batch([(1, 5)], 16, 1, 64)
    t = dict(cu_rows=bt.cu, lens=bt.lens, page_table=bt.table, k_codes=bt.k, v_codes=bt.v, k_scales=bt.ks, v_scales=bt.vs)
    x = torch.zeros(1, 3 * 64, dtype=torch.bfloat16)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="qkv: device tensor"):
        mq.mq_rope_kv_append(x, None, q_out=q, **t)
    with pytest.raises(ValueError, match="q: device tensor"):
        mq.mq_kv_attention(q, out=q, ws=bt.k, max_q=1, max_len=5, scale=0.1, **t)
    with pytest.raises(ValueError, match="x: device tensor"):
        mq.mq_linear_w4a16(x, bt.k, bt.k, bt.ks, 1, x)
    with pytest.raises(ValueError, match="x: tensor expected"):
        mq.mq_linear_w4a16(None, bt.k, bt.k, bt.ks, 1, x)
    with pytest.raises(TypeError):
        mq.mq_linear_w4a16(x, bt.k, bt.k, bt.ks, "N", x)


def test_the_header_s_limit_of_rows(L):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "mq.h")).read()
    assert int(re.search(r"#define MQ_LINEAR_W4A16_MAX_M (\d+)", text).group(1)) == 64


# -- the rotary table ----------------------------------------------------------------

def _table(positions, rot, theta, f=None, size=1.0):
    out = torch.empty(positions, rot)
    for p in range(positions):
        for j in range(rot // 2):
            w = theta ** (-2 * j / rot) if f is None else f(j)
            out[p, j], out[p, rot // 2 + j] = math.cos(p * w) * size, math.sin(p * w) * size
    return out


def test_rope_table():
    # half a step of binary32 of values up to 1, and an angle's error in 64 bits
    close = lambda a, b: bool(((a - b).abs() <= 2.0 ** -24 + 1e-12).all())
    assert close(mq.rope_table(40, 16, 1e4, device="cpu"), _table(40, 16, 1e4))
    assert close(mq.rope_table(40, 16, 1e4, dict(kind="linear", factor=4.0), device="cpu"),
                 _table(40, 16, 1e4, lambda j: 1e4 ** (-2 * j / 16) / 4))
    with pytest.raises(ValueError):
        mq.rope_table(4, 15, device="cpu")
    with pytest.raises(ValueError):
        mq.rope_table(4, 16, scaling=dict(kind="other", factor=2.0), device="cpu")


def test_rope_table_yarn():
    """Fast pairs keep their frequency, slow ones are divided, the blend runs from one to the other."""
    L0, s, rot, theta = 4096, 8.0, 64, 1e4
    t = mq.rope_table(2, rot, theta, dict(kind="yarn", factor=s, original=L0), device="cpu").double()
    size = 0.1 * math.log(s) + 1
    f = torch.atan2(t[1, rot // 2:], t[1, :rot // 2])
    plain = torch.tensor([theta ** (-2 * j / rot) for j in range(rot // 2)], dtype=torch.float64)
    turns = plain * L0 / (2 * math.pi)
    # atan2 of two roundings of 2^-24 each
    assert (t[0, :rot // 2] - size).abs().max() <= 2.0 ** -23
    ratio = f / plain
    tol = 2.0 ** -22 / plain
    assert (ratio[turns > 40] - 1).abs().le(tol[turns > 40]).all()
    assert (ratio[turns < 0.8] - 1 / s).abs().le(tol[turns < 0.8]).all()
    assert (ratio[1:] <= ratio[:-1] + tol[1:] + tol[:-1]).all()


# -- the tests' plain forms -----------------------------------------------------------

def test_page_exponent():
    """Least e with amax <= 448 2^e."""
    g = torch.Generator().manual_seed(0)
    xs = [448.0, 448.0001, 447.9, 1.0, 1.75, 1.7500001, 2.0 ** -60, 3.3e38, 0.0] + torch.randn(200, generator=g).abs().tolist()
    for x in xs:
        e = kv.exponent(x)
        assert kv.E_MIN <= e <= kv.E_MAX
        if x > 448.0 * 2.0 ** kv.E_MAX:
            assert e == kv.E_MAX
        else:
            assert x <= 448.0 * 2.0 ** e
            assert e == kv.E_MIN or x > 448.0 * 2.0 ** (e - 1)


def test_a_planted_mistake_is_seen():
    """The comparison fails for an output that is off by one bf16 step, and for a row of another sequence."""
    bt = kv.Batch([(3, 20), (2, 9)], 16, 1, 64, seed=1).fill()
    q = torch.randn(bt.T, 2, 64).bfloat16()
    want, bound = kv.attention_plain(bt, q, 0.125)
    got = want.bfloat16()
    kv.close_to(got, want, bound)
    big = torch.argmax(want.abs())
    bad = got.clone().view(-1)
    bad[big] = bad[big] * (1 + 2.0 ** -5)
    with pytest.raises(AssertionError):
        kv.close_to(bad.view(got.shape), want, bound)
    with pytest.raises(AssertionError):
        kv.close_to(got[[3, 1, 2, 0, 4]], want, bound)


def test_plain_attention_by_hand():
    """Two keys, exact numbers: weights 1/2 and 1/2, then 1 and 0."""
    bt = kv.Batch([(2, 2)], 16, 1, 64, seed=2)
    p = int(bt.table[0, 0])
    k = torch.zeros(2, 64)
    v = torch.zeros(2, 64)
    v[0, :], v[1, :] = 2.0, 4.0
    bt.k[p, 0, :2], bt.v[p, 0, :2] = kv.e4m3(k).view(torch.uint8), kv.e4m3(v).view(torch.uint8)
    bt.ks[p], bt.vs[p] = 1.0, 0.5
    q = torch.ones(2, 1, 64).bfloat16()
    out, _ = kv.attention_plain(bt, q, 1.0)
    assert out[0, 0, 0] == 1.0 and out[1, 0, 0] == 1.5
