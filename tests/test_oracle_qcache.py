"""The quantised history cache in the oracle, and the library's refusals, without a GPU."""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from gen.synth import bf16_round


def _bf16(x):
    return bf16_round(np.asarray(x, np.float32)).astype(np.float64)


def _heads(seed, n=400):
    r = np.random.default_rng(seed)
    x = r.standard_normal((n, 64)) * np.exp(r.uniform(-60, 60, (n, 1)))
    x[0] = 0.0
    x[1, 1:] = 0.0
    x[2] = 3.3895313892515355e38  # the largest bf16
    x[3] = 1e-39                  # below the smallest scale
    x[4] = 7.0
    x[5] = 7.0 * 33 * np.where(np.arange(64) % 2, 1, -1)  # a / 7 halfway between two scales
    x[6, :] = np.arange(64) + 64.5  # halves of the 8-bit step
    x[7] = 127.0
    x[8] = 127.5
    return _bf16(x)


@pytest.mark.parametrize("bits", [8, 4])
def test_codes_scales_and_error(bits):
    x = _heads(1)
    c, s = oracle.qcache_quantise(x, bits)
    most = 127 if bits == 8 else 7
    assert np.abs(c).max() <= most
    a = np.abs(x).max(-1)
    # the value is a bf16 number: code and scale have at most 8 significant bits together
    v = c * s[:, None]
    assert np.array_equal(_bf16(v), v)
    # nearest code: half a step, or what the clamp leaves of the largest magnitude
    inside = (s > 2.0 ** -126) & (a < 1e38)
    step = np.abs(x - v)[inside] / s[inside][:, None]
    assert step.max() <= 0.5
    # the scale spends its range: one bit at most in 8 bits, 1/32 in 4 bits
    big = inside & (a > 0)
    need = a[big] / most
    if bits == 8:
        assert np.all(need <= s[big]) and np.all(s[big] < 2 * need)
        assert np.all(np.frexp(s[big])[0] == 0.5)
    else:
        assert np.all(np.abs(s[big] - need) <= need / 32)


def test_not_finite_heads_read_back_as_nan():
    x = np.ones((3, 64))
    x[0, 5] = np.inf
    x[1, 63] = np.nan
    for bits in (8, 4):
        v = oracle.qcache_values(x, bits)
        assert np.isnan(v[:2]).all() and np.isfinite(v[2]).all()


@pytest.mark.parametrize("H,bits", [(1, 8), (3, 4), (4, 4), (8, 8), (9, 4), (64, 8)])
def test_row_bytes_match_the_library(H, bits):
    from generative_ranking_recommendation_b200 import genrank as G
    from generative_ranking_recommendation_b200.csrc import build

    build.build()
    fmt = G.QCACHE_INT8 if bits == 8 else G.QCACHE_INT4
    k = np.ones((2, H, 64))
    rows = oracle.qcache_rows(k, -k, np.array([1, 2]), np.array([5, 1 << 40]), bits)
    assert rows.shape[1] == G.qcache_row_bytes(H, 64, fmt)
    assert rows.shape[1] % 32 == 16


def test_attention_equals_the_cached_oracle():
    r = np.random.default_rng(3)
    H, lens, cands = 2, [5, 0, 9], [2, 1, 3]
    n, C = sum(lens), sum(cands)
    k, v = r.standard_normal((2, n, H, 64))
    q, kc, vc = r.standard_normal((3, C, H, 64))
    hoff, coff = np.concatenate([[0], np.cumsum(lens)]), np.concatenate([[0], np.cumsum(cands)])
    pos = np.concatenate([np.arange(1, x + 1) for x in lens])
    ts = np.concatenate([np.sort(r.integers(0, 1000, x)) for x in lens])
    tc = r.integers(1000, 1100, C)
    sp = oracle.alibi_slopes(H)
    args = (sp, sp / 3600, 0.125)
    want = oracle.attention_fwd_cached(q, kc, vc, coff, k, v, hoff, pos, ts, tc, *args)
    got = oracle.attention_fwd_qcached(q, kc, vc, coff, k, v, hoff[:-1], lens, pos, ts, tc, *args)
    assert np.max(np.abs(got[0] - want[0])) <= 1e-12 and np.max(np.abs(got[1] - want[1])) <= 1e-12


@pytest.fixture(scope="module")
def L():
    from generative_ranking_recommendation_b200 import genrank as G
    from generative_ranking_recommendation_b200.csrc import build

    build.build()
    return G.lib()


P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: every call below fails its host checks


def test_write_and_read_refusals(L):
    def call(read=False, **kw):
        a = dict(B=2, T=10, off=FAKE, len=None, k=FAKE, v=FAKE, stride=256, H=4, dh=64, dtype=1,
                 pos=FAKE, ts=FAKE, fmt=1, cache=FAKE, R=100, rows=FAKE, err=FAKE)
        a.update(kw)
        if read:
            return L.genrank_qcache_read(a["B"], a["T"], a["off"], a["len"], a["cache"], a["R"],
                                         a["rows"], a["H"], a["dh"], a["fmt"], a["k"], a["v"],
                                         a["stride"], a["dtype"], a["pos"], a["ts"], a["err"], None)
        return L.genrank_qcache_append(a["B"], a["T"], a["off"], a["len"], a["k"], a["v"],
                                       a["stride"], a["H"], a["dh"], a["dtype"], a["pos"], a["ts"],
                                       a["fmt"], a["cache"], a["R"], a["rows"], a["err"], None)

    for read in (False, True):
        assert call(read, B=0) == 1
        assert call(read, T=-1) == 1
        assert call(read, R=-1) == 1
        assert call(read, off=None) == 1
        assert call(read, rows=None) == 1
        assert call(read, err=None) == 1
        assert call(read, k=None) == 1
        assert call(read, v=P(0x10008)) == 1
        assert call(read, cache=None) == 1
        assert call(read, cache=P(0x10004)) == 1
        assert call(read, fmt=2) == 1
        assert call(read, dtype=5) == 1
        assert call(read, stride=255) == 1
        assert call(read, stride=260) == 1  # bf16: 520 bytes, not a multiple of 16
        assert call(read, dh=32, stride=256) == 2
        assert call(read, H=65, stride=65 * 64) == 2
        assert call(read, T=1 << 31) == 2
        assert call(read, T=0, k=None, v=None, cache=None, pos=None, ts=None) == 0  # nothing to do
    assert call(pos=None) == 1
    assert call(ts=None) == 1


def test_attention_refusals(L):
    sp = (ctypes.c_float * 64)(*([0.5] * 64))
    bad = (ctypes.c_float * 64)(*([0.5] * 3 + [float("nan")] * 61))
    neg = (ctypes.c_float * 64)(*([-1.0] * 64))

    def call(**kw):
        a = dict(B=2, C=10, off=FAKE, max_cand=5, q=FAKE, k=FAKE, v=FAKE, stride=768, cache=FAKE,
                 R=100, rows=FAKE, len=FAKE, max_len=2000, ts=FAKE, fmt=1, H=4, dh=64, sp=sp, st=sp,
                 scale=0.125, dtype=1, o=FAKE, ostride=256, lse=None, ws=FAKE, wsb=1 << 30, err=FAKE)
        a.update(kw)
        return L.genrank_attn_fwd_qcached(
            a["B"], a["C"], a["off"], a["max_cand"], a["q"], a["k"], a["v"], a["stride"],
            a["cache"], a["R"], a["rows"], a["len"], a["max_len"], a["ts"], a["fmt"], a["H"],
            a["dh"], ctypes.cast(a["sp"], P), ctypes.cast(a["st"], P), a["scale"], a["dtype"],
            a["o"], a["ostride"], a["lse"], a["ws"], a["wsb"], a["err"], None)

    for kw in (dict(B=0), dict(C=-1), dict(off=None), dict(q=None), dict(k=P(0x10008)), dict(o=None),
               dict(o=P(0x10002)), dict(ts=None), dict(rows=None), dict(len=None), dict(err=None),
               dict(cache=None), dict(cache=P(0x10008)), dict(fmt=3), dict(scale=0.0),
               dict(scale=math.inf), dict(stride=100), dict(stride=260), dict(ostride=252),
               dict(max_cand=-1), dict(max_len=-1), dict(st=bad), dict(sp=neg), dict(dtype=9), dict(R=-1)):
        assert call(**kw) == 1, kw
    assert call(dtype=0) == 2  # fp32 candidates
    assert call(dh=128, stride=1536, ostride=512) == 2
    assert call(H=65, stride=3 * 65 * 64, ostride=65 * 64) == 2
    assert call(max_len=(1 << 30) + 1) == 2
    assert call(ws=None) == 3
    assert call(wsb=16) == 3
    assert call(ws=P(0x10004)) == 3
    assert call(C=0, q=None, k=None, v=None, o=None, ts=None, ws=None, wsb=0) == 0


def test_workspace_and_row_sizes(L):
    assert L.genrank_qcache_row_bytes(8, 64, 0) == 1072 and L.genrank_qcache_row_bytes(8, 64, 1) == 560
    for args in ((0, 64, 0), (65, 64, 0), (8, 32, 0), (8, 64, 2)):
        assert L.genrank_qcache_row_bytes(*args) == 0
    ws = L.genrank_attn_qcached_workspace_size
    assert ws(1, 1, 8, 64, 1, 4096) > 0      # few blocks: ranges of the history are joined
    assert ws(4096, 4096, 8, 64, 1, 480) == 0
    assert ws(1, 1, 8, 64, 1, 0) == 0
    # the largest bounds
    assert ws(1, 1, 8, 64, 1, 1 << 30) > 0 and ws(1, 1, 8, 64, 1, (1 << 30) + 1) == 0
    assert ws(2**31 - 1, 1, 64, 64, 2**31 - 1, 1 << 30) == 0
    assert ws(1, 1, 8, 64, 2**31 - 1, 1 << 30) == 0
    for args in ((0, 1, 8, 64, 1, 10), (1, -1, 8, 64, 1, 10), (1, 1, 8, 32, 1, 10), (1, 1, 65, 64, 1, 10),
                 (1, 1, 8, 64, -1, 10), (1, 1, 8, 64, 1, -1)):
        assert ws(*args) == 0


def test_python_refusals():
    """The binding refuses tensors of the wrong type, shape or place before any call."""
    from generative_ranking_recommendation_b200 import genrank as G

    with pytest.raises(G.GenRankError):
        G.qcache_row_bytes(8, 32, G.QCACHE_INT8)
    cpu = torch.zeros(4, 560, dtype=torch.uint8)
    k = torch.zeros(4, 512, dtype=torch.bfloat16)
    off, rows = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    pos, ts, err = torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(G.GenRankError):  # host tensors
        G.qcache_append(off, None, k, k, 512, 8, 64, pos, ts, cpu, rows, G.QCACHE_INT4, err)
    with pytest.raises(G.GenRankError):  # rows of another format
        G.qcache_append(off, None, k, k, 512, 8, 64, pos, ts, cpu, rows, G.QCACHE_INT8, err)
