"""The quantised history cache on a GPU: rows written to it bit for bit against the oracle,
rows read back, and candidate attention over it against the float64 oracle on the values the
cache stands for.

Tolerances.  A cache value is exact, so append and read have none.  Attention, with
A = sum_j p_j |v_j| and S = max_j scale sum_i |q_i k_i|:
  O    2^-8 |O| (rounding to bf16) + A (2^-11 (each p_j rounded to fp16) + 2 e) + n 2^-30 max |v|
       (p_j below fp16's normal range), e the relative error of a p_j:
  e    2^-18 S (fp32 sums of 64 products and their scale, log2 units) + 2^-19 (the exponential, its
       argument of at most 2^5 where p_j matters, the sums)
  LSE  e + 2^-22 (|LSE| + |the row's time term|)
"""

import math

import numpy as np
import pytest
import torch

import oracle
from gen.synth import bf16_round

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    from generative_ranking_recommendation_b200 import genrank
    from generative_ranking_recommendation_b200.csrc import build

    build.build()
    genrank.lib()
    return genrank


def _dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def _fmt(G, bits):
    return G.QCACHE_INT8 if bits == 8 else G.QCACHE_INT4


def _bf16(x):
    return bf16_round(np.asarray(x, np.float32))


def _kv(r, n, H, spread=1.0):
    """Keys or values [n, H, 64] in bf16: heads of unequal scale."""
    return _bf16(r.standard_normal((n, H, 64)) * np.exp2(r.uniform(-spread, spread, (n, H, 1))))


# ------------------------------------------------------------------------------------------
# writing
# ------------------------------------------------------------------------------------------

def _append(G, k, v, pos, ts, off, length, rows, R, bits, dtype=torch.bfloat16, pad=16, cache=None, fill=0x5A):
    T, H = k.shape[:2]
    d = H * 64
    wide = torch.zeros(T, 2 * d + pad, dtype=dtype, device="cuda")
    wide[:, :d] = _dev(k.reshape(T, d))
    wide[:, d:2 * d] = _dev(v.reshape(T, d))
    if cache is None:
        cache = torch.full((R, G.qcache_row_bytes(H, 64, _fmt(G, bits))), fill, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    G.qcache_append(_dev(off, torch.int32), None if length is None else _dev(length, torch.int32), wide, wide[:, d:],
                    2 * d + pad, H, 64, _dev(pos, torch.int32), _dev(ts, torch.int64), cache,
                    _dev(rows, torch.int64), _fmt(G, bits), err)
    return cache, G.check_error(err)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [1, 3, 8, 9, 16, 64])
def test_append_bytes(G, bits, dtype, H):
    r = np.random.default_rng(H)
    seg, length, gap = [3, 0, 40, 1, 17], [2, 0, 33, 1, 17], [0, 2, 1, 0, 3]
    off = np.concatenate([[0], np.cumsum(seg)])
    T = int(off[-1]) + 4  # rows of nobody behind the last user
    shape = (T, H, 64)
    x = [r.standard_normal(shape) * np.exp2(r.uniform(-20, 20, (T, H, 1))) for _ in range(2)]
    x = [np.asarray(a, np.float32) for a in x] if dtype == torch.float32 else [_bf16(a) for a in x]
    pos = r.integers(0, 1000, T)
    ts = r.integers(-(1 << 40), 1 << 40, T)
    rows = np.zeros(5, np.int64)
    at = 1
    for u in range(5):
        rows[u] = at + gap[u]
        at = rows[u] + length[u]
    R = int(at) + 2
    cache, code = _append(G, x[0], x[1], pos, ts, off, length, rows, R, bits, dtype)
    assert code == 0
    want = np.full((R, cache.shape[1]), 0x5A, np.uint8)
    for u in range(5):
        s = slice(int(off[u]), int(off[u]) + length[u])
        want[rows[u]:rows[u] + length[u]] = oracle.qcache_rows(_bf16(x[0][s]), _bf16(x[1][s]), pos[s], ts[s], bits)
    assert np.array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("bits", [8, 4])
def test_append_special_heads(G, bits):
    """Zero heads, the largest and the smallest bf16, halves of a step, every 8-bit mantissa as
    the maximum, infinities and NaN (whose head alone is lost)."""
    r = np.random.default_rng(2)
    k = _kv(r, 300, 2)
    k[0] = 0.0
    k[1, 0] = 3.3895313892515355e38
    k[1, 1] = -3.3895313892515355e38
    k[2] = 1e-39
    k[3, 0] = np.arange(64) + 64.5
    k[3, 1] = (np.arange(64) - 31.5) * 7 / 31.5 * 3
    k[4, 0, 7] = np.inf
    k[5, 1, 8] = -np.inf
    k[6, 0, 9] = np.nan
    for i in range(128):
        k[10 + i] = np.exp2(float(i % 7)) * (128 + i) / 128 * (np.arange(128).reshape(2, 64) - 64) / 64
        k[10 + i, :, 0] = np.exp2(float(i % 7)) * (128 + i) / 128
    k = _bf16(k)
    v = k[::-1].copy()
    n = len(k)
    pos, ts = np.arange(n), np.arange(n)
    cache, code = _append(G, k, v, pos, ts, [0, n], None, [0], n, bits)
    assert code == 0
    assert np.array_equal(cache.cpu().numpy(), oracle.qcache_rows(k, v, pos, ts, bits))


def test_append_layout_errors(G):
    """Users whose ranges leave the arrays or meet the next user's are left out and flagged."""
    r = np.random.default_rng(4)
    k = _kv(r, 12, 1)
    pos, ts = np.arange(12), np.arange(12)

    def run(off, length, rows, R=40):
        cache, code = _append(G, k, k, pos, ts, off, length, rows, R, 8)
        return (cache.cpu().numpy() != 0x5A).any(-1).nonzero()[0].tolist(), code

    ok = [0, 1, 2, 3, 10, 11, 12, 13, 20, 21, 22, 23]
    assert run([0, 4, 8, 12], None, [0, 10, 20]) == (ok, 0)
    assert run([0, 4, 8, 12], None, [0, 10, 37]) == (ok[:8], G.DERR["LAYOUT"])       # past the cache
    assert run([0, 4, 8, 12], None, [-1, 10, 20]) == (ok[4:], G.DERR["LAYOUT"])
    assert run([0, 4, 8, 12], None, [8, 10, 20]) == (ok[4:], G.DERR["LAYOUT"])       # meets the next user
    assert run([0, 4, 8, 12], [4, 5, 4], [0, 10, 20]) == (ok[:4] + ok[8:], G.DERR["LAYOUT"])  # longer than its rows
    assert run([0, 4, 8, 12], [4, -1, 4], [0, 10, 20]) == (ok[:4] + ok[8:], G.DERR["LAYOUT"])
    assert run([0, 4, 8, 13], None, [0, 10, 20]) == (ok[:8], G.DERR["LAYOUT"])       # past the token rows
    assert run([0, 4, 4, 8], None, [0, 10, 10]) == (ok[:8], 0)                       # a user without rows
    assert run([0, 4, 4, 8], None, [0, 3, 10])[1] == G.DERR["LAYOUT"]                # ... in its place all the same


def test_rows_beyond_32_bit_offsets(G):
    """A row whose byte offset passes 2^32, written and read back."""
    rb = G.qcache_row_bytes(8, 64, G.QCACHE_INT8)
    R = (1 << 32) // rb + 100
    r = np.random.default_rng(5)
    k, v = _kv(r, 3, 8), _kv(r, 3, 8)
    cache = torch.empty(R, rb, dtype=torch.uint8, device="cuda")
    cache[0] = 0
    pos, ts = [5, 6, 7], [1 << 33, 1 << 34, 1 << 35]
    cache, code = _append(G, k, v, pos, ts, [0, 3], None, [R - 3], R, 8, cache=cache)
    assert code == 0 and not cache[0].any()
    assert np.array_equal(cache[R - 3:].cpu().numpy(), oracle.qcache_rows(k, v, pos, ts, 8))
    out = torch.empty(2, 3, 512, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    G.qcache_read(_dev([0, 3], torch.int32), None, cache, _dev([R - 3], torch.int64), out[0], out[1], 512, 8, 64,
                  None, None, G.QCACHE_INT8, err)
    assert G.check_error(err) == 0
    for side, x in enumerate((k, v)):
        assert np.array_equal(out[side].float().cpu().numpy().reshape(3, 8, 64), oracle.qcache_values(x, 8))
    # and scored against
    q = _bf16(r.standard_normal((1, 3, 8, 64)))
    o, lse, code = _score(G, q, [0, 1], cache, [R - 3], [3], [1 << 36], 8, 8)
    assert code & G.DERR["POS_RANGE"]  # positions 5..7 of a history of three
    cache[R - 3:] = _dev(oracle.qcache_rows(k, v, [1, 2, 3], ts, 8))
    _compare(G, q, [0, 1], cache, [R - 3], [3], [1 << 36], 8, 8,
             values=(oracle.qcache_values(k, 8), oracle.qcache_values(v, 8), [1, 2, 3], ts), base=R - 3)


# ------------------------------------------------------------------------------------------
# reading back
# ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [1, 5, 8, 16])
def test_read_back(G, bits, dtype, H):
    """Users in any order, one of them twice, some rows only; other output rows left alone."""
    r = np.random.default_rng(H)
    N = 60
    k, v = _kv(r, N, H, 30.0), _kv(r, N, H, 30.0)
    pos, ts = r.integers(0, 99, N), r.integers(0, 1 << 40, N)
    cache = _dev(oracle.qcache_rows(k, v, pos, ts, bits))
    rows, length, seg = [40, 0, 7, 40], [20, 5, 0, 3], [21, 5, 2, 3]
    off = np.concatenate([[1], 1 + np.cumsum(seg)])
    T, d = int(off[-1]) + 3, H * 64
    stride = d + 16
    out = torch.full((2, T, stride), -7.0, dtype=dtype, device="cuda")
    po = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    to = torch.full((T,), -7, dtype=torch.int64, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    G.qcache_read(_dev(off, torch.int32), _dev(length, torch.int32), cache, _dev(rows, torch.int64), out[0], out[1],
                  stride, H, 64, po, to, _fmt(G, bits), err)
    assert G.check_error(err) == 0
    want = np.full((2, T, stride), -7.0)
    wp, wt = np.full(T, -7), np.full(T, -7)
    for u in range(4):
        d0, s = slice(int(off[u]), int(off[u]) + length[u]), slice(rows[u], rows[u] + length[u])
        want[0, d0, :d] = oracle.qcache_values(k[s], bits).reshape(-1, d)
        want[1, d0, :d] = oracle.qcache_values(v[s], bits).reshape(-1, d)
        wp[d0], wt[d0] = pos[s], ts[s]
    assert np.array_equal(out.double().cpu().numpy(), want)
    assert np.array_equal(po.cpu().numpy(), wp) and np.array_equal(to.cpu().numpy(), wt)


def test_read_layout_errors(G):
    cache = _dev(oracle.qcache_rows(np.ones((4, 1, 64)), np.ones((4, 1, 64)), range(4), range(4), 4))
    for rows, off, length in (([3], [0, 2], None), ([-1], [0, 2], None), ([0], [0, 9], None), ([0], [0, 2], [3])):
        out = torch.full((2, 4, 64), -7.0, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        G.qcache_read(_dev(off, torch.int32), None if length is None else _dev(length, torch.int32), cache,
                      _dev(rows, torch.int64), out[0], out[1], 64, 1, 64, None, None, G.QCACHE_INT4, err)
        assert G.check_error(err) == G.DERR["LAYOUT"]
        assert (out == -7.0).all()


# ------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------

def _score(G, qkv, coff, cache, rows, lens, tc, H, bits, slopes=None, poison=True, extra=0, max_cand=None,
           max_len=None, pad=8, lse=True):
    """qkv: [3 (q, k, v), C, H, 64] or [C, 3, H, 64] with C = 1; outputs as float64 [C + extra, H, 64], [H, C + extra]."""
    qkv = np.asarray(qkv)
    if qkv.shape[0] != 3:
        qkv = qkv.transpose(1, 0, 2, 3)
    C, d = qkv.shape[1], H * 64
    stride = 3 * d + pad
    x = torch.zeros(C, stride, dtype=torch.bfloat16, device="cuda")
    for i in range(3):
        x[:, i * d:(i + 1) * d] = _dev(qkv[i].reshape(C, d))
    B = len(rows)
    coff = np.asarray(coff)
    max_cand = int(np.max(np.diff(coff))) if max_cand is None else max_cand
    max_len = int(np.max(lens)) if max_len is None else max_len
    need = G.attn_qcached_workspace_size(B, C + extra, H, 64, max_cand, max_len)
    ws = torch.full((max(need, 16),), 0xFF if poison else 0, dtype=torch.uint8, device="cuda")
    o = torch.full((C + extra, d + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    ls = torch.full((H, C + extra), float("nan"), dtype=torch.float32, device="cuda") if lse else None
    if extra:
        x = torch.cat([x, torch.full((extra, stride), float("nan"), dtype=torch.bfloat16, device="cuda")])
        tc = list(tc) + [0] * extra
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sp, st = slopes or G.alibi_slopes(H)
    G.attn_fwd_qcached(_dev(coff, torch.int32), max_cand, x, x[:, d:], x[:, 2 * d:], stride, cache,
                       _dev(rows, torch.int64), _dev(lens, torch.int32), max_len, _dev(tc, torch.int64), H, 64, sp, st,
                       0.125, o, d + pad, ls, ws if need else None, _fmt(G, bits), err, C=C + extra)
    code = G.check_error(err)
    assert torch.isnan(o[:, d:]).all()  # between the rows' ends and the stride
    return (o[:, :d].double().cpu().numpy().reshape(C + extra, H, 64),
            None if ls is None else ls.double().cpu().numpy(), code)


def _compare(G, qkv, coff, cache, rows, lens, tc, H, bits, values, base=0, slopes=None, **kw):
    """values: (k, v, pos, ts) that the cache stands for, from cache row `base` on."""
    o, lse, code = _score(G, qkv, coff, cache, rows, lens, tc, H, bits, slopes=slopes, **kw)
    assert code == 0
    qkv = np.asarray(qkv, np.float64)
    if qkv.shape[0] != 3:
        qkv = qkv.transpose(1, 0, 2, 3)
    sp, st = slopes or G.alibi_slopes(H)
    k, v, pos, ts = values
    want, wl, A, S = oracle.attention_fwd_qcached(*qkv, coff, k, v, np.asarray(rows) - base, lens, pos, ts, tc, sp, st, 0.125)
    C = len(want)
    extra = len(o) - C
    assert np.isnan(o[C:]).all() and (lse is None or np.isnan(lse[:, C:]).all())
    o = o[:C]
    e = 2.0 ** -18 * S + 2.0 ** -19  # [H, C]
    n = max(lens) if len(lens) else 0
    top = max(np.abs(qkv[2]).max(), np.abs(v).max() if len(v) else 0.0)
    tol = 2.0 ** -8 * np.abs(want) + A * (2.0 ** -11 + 2 * e.T[:, :, None]) + n * 2.0 ** -30 * top
    assert np.all(np.abs(o - want) <= tol), np.max(np.abs(o - want) / tol)
    if lse is not None:
        row = np.zeros(C)
        for u in range(len(rows)):
            c = slice(coff[u], coff[u + 1])
            if coff[u + 1] > coff[u]:
                row[c] = np.abs(np.asarray(tc)[c] - np.asarray(tc)[coff[u]])
        tol = e + 2.0 ** -22 * (np.abs(wl) + np.asarray(st)[:, None] * row)
        assert np.all(np.abs(lse[:, :C] - wl) <= tol), np.max(np.abs(lse[:, :C] - wl) / tol)
    return o, lse, extra


def _batch(seed, users, H, bits, spread=1.0, tc_spread=0, qscale=1.0, slack=3, order=None):
    """Users (n, m) with their rows somewhere in a cache whose other rows are noise."""
    r = np.random.default_rng(seed)
    B = len(users)
    lens, cands = [n for n, _ in users], [m for _, m in users]
    order = r.permutation(B) if order is None else order
    rows, at = np.zeros(B, np.int64), 2
    for u in order:
        rows[u] = at
        at += lens[u] + int(r.integers(0, slack + 1))
    R = at + 2
    k, v = _kv(r, R, H, spread), _kv(r, R, H, spread)
    pos, ts = np.zeros(R, np.int64), np.zeros(R, np.int64)
    noise = np.ones(R, bool)
    for u in range(B):
        s = slice(rows[u], rows[u] + lens[u])
        pos[s] = np.arange(1, lens[u] + 1)
        gaps = np.where(r.random(lens[u]) < 0.5, r.exponential(30.0, lens[u]), r.exponential(3600.0, lens[u]))
        ts[s] = 1_700_000_000 + np.cumsum(gaps).astype(np.int64)
        noise[s] = False
    rb = oracle.qcache_rows(k, v, pos, ts, bits)
    rb[noise] = r.choice(np.array([0x7F, 0x80, 0xFF, 0xC0], np.uint8), (int(noise.sum()), rb.shape[1]))
    coff = np.concatenate([[0], np.cumsum(cands)])
    C = int(coff[-1])
    qkv = np.stack([_bf16(qscale * r.standard_normal((C, H, 64))), _kv(r, C, H, spread), _kv(r, C, H, spread)])
    tc = np.zeros(C, np.int64)
    for u in range(B):
        last = ts[rows[u] + lens[u] - 1] if lens[u] else 1_700_000_000
        m = cands[u]
        tc[coff[u]:coff[u + 1]] = last + 7 + (r.integers(0, tc_spread + 1, m) if tc_spread else 0)
    values = (oracle.qcache_values(k, bits), oracle.qcache_values(v, bits), pos, ts)
    return dict(qkv=qkv, coff=coff, cache=rb, rows=rows, lens=lens, tc=tc, H=H, bits=bits), values


def _check(G, batch, values, **kw):
    b = dict(batch)
    b["cache"] = _dev(b["cache"])
    return _compare(G, b.pop("qkv"), b.pop("coff"), b.pop("cache"), b.pop("rows"), b.pop("lens"), b.pop("tc"),
                    b.pop("H"), b.pop("bits"), values, **kw)


# (history, candidates): empty histories, users without candidates, lengths around the tile of 32
# rows, candidates around the tiles of 8, 16 and 32
SMALL = [(0, 1), (1, 1), (31, 2), (32, 3), (33, 8), (0, 0), (64, 0), (65, 7), (127, 5), (480, 4), (300, 6)]
MIDDLE = SMALL + [(40, 9), (33, 16), (0, 15)]
LARGE = MIDDLE + [(100, 31), (63, 32), (96, 33), (5, 70), (480, 129)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("users", [SMALL, MIDDLE, LARGE], ids=["small", "middle", "large"])
@pytest.mark.parametrize("H", [1, 2, 5, 8, 9, 16])
def test_attention(G, bits, users, H):
    _check(G, *_batch(H, users, H, bits, tc_spread=5000), extra=3)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("most", [0, 1, 32, 33, 64, 65, 96, 97])
def test_short_histories(G, bits, most):
    """Blocks that stage no more tiles than the bound needs, up to all of them."""
    lens = [n for n in (0, 1, 31, 32, 33, 63, 64, 65, 95, 96, 97) if n <= most]
    users = [(n, 1 + (3 * i) % 11) for i, n in enumerate(lens * 8)]
    _check(G, *_batch(most, users, 9, bits), extra=1)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("n,m,H", [(1, 1, 8), (480, 1, 8), (1000, 8, 3), (4097, 1, 8), (2051, 33, 2), (9000, 2, 17),
                                   (64, 1, 64), (65, 300, 1)])
def test_one_user_in_ranges(G, bits, n, m, H):
    """One user: the history is cut into ranges that are joined."""
    _check(G, *_batch(n, [(n, m)], H, bits))


def test_many_users(G):
    """More blocks than fit at once, 4 and 8 bits, no workspace."""
    r = np.random.default_rng(9)
    users = [(int(r.integers(0, 90)), int(r.integers(0, 4))) for _ in range(2000)]
    batch, values = _batch(9, users, 2, 4)
    assert G.attn_qcached_workspace_size(2000, len(batch["tc"]), 2, 64, 3, 89) == 0
    _check(G, batch, values)


@pytest.mark.parametrize("bits", [8, 4])
def test_many_users_of_unequal_length(G, bits):
    """More blocks than fit at once, the longer histories first: lengths on both sides of half the
    bound, and exactly half."""
    r = np.random.default_rng(10)
    users = [(int(r.choice([0, 1, 299, 300, 301, 600])), int(r.integers(0, 3))) for _ in range(500)]
    batch, values = _batch(10, users, 2, bits)
    _check(G, batch, values, max_len=600)
    _, _, code = _score(G, **dict(batch, cache=_dev(batch["cache"])), max_len=599)
    assert code == G.DERR["LAYOUT"]


@pytest.mark.parametrize("bits", [8, 4])
def test_unequal_magnitudes(G, bits):
    """V scales over 2^+-20 within a history, and scores of some hundreds: the running maximum
    and the range of P move often; a candidate's own score far above and far below the rest."""
    batch, values = _batch(11, [(200, 8), (333, 5), (70, 3)], 4, bits, spread=20.0, qscale=1e-4)
    _check(G, batch, values)
    batch, values = _batch(12, [(200, 8), (333, 20), (70, 3)], 4, bits, qscale=60.0)
    batch["qkv"][1, ::3] *= 8.0
    batch["qkv"][1, 1::3] *= -8.0
    _check(G, batch, values)


def test_extreme_magnitudes_of_q(G):
    """q of 2^100 against keys of 2^-100, and the other way round; a zero q; candidates of one
    tile a factor 2^12 apart."""
    for up in (100, -100):
        batch, _ = _batch(13, [(77, 4)], 2, 4)
        r = np.random.default_rng(1)
        n, R = 77, len(batch["cache"])
        k, v = _kv(r, R, 2) * np.float32(2.0 ** -up), _kv(r, R, 2)
        pos, ts = np.zeros(R, np.int64), np.zeros(R, np.int64)
        s = slice(batch["rows"][0], batch["rows"][0] + n)
        pos[s], ts[s] = np.arange(1, n + 1), batch["tc"][0] - 5
        batch["cache"] = oracle.qcache_rows(k, v, pos, ts, 4)
        batch["qkv"][0] *= np.float32(2.0 ** up)
        batch["qkv"][0, 1] = 0.0
        batch["qkv"][0, 2] *= np.float32(2.0 ** -12)
        batch["qkv"][1] *= np.float32(2.0 ** -up)
        _check(G, batch, (oracle.qcache_values(k, 4), oracle.qcache_values(v, 4), pos, ts))


@pytest.mark.parametrize("slopes", ["none", "position", "time"])
def test_slopes(G, slopes):
    H = 3
    sp = [0.0] * H if slopes != "position" else [2.0, 0.01, 0.0]
    st = [0.0] * H if slopes != "time" else [1.0, 1e-5, 1e-9]
    batch, values = _batch(14, [(150, 6), (31, 2), (0, 1)], H, 8, tc_spread=100000)
    _check(G, batch, values, slopes=(sp, st))


def test_far_times(G):
    """Gaps of centuries between the interactions and the request."""
    batch, values = _batch(15, [(60, 3)], 2, 4)
    values[3][values[3] > 0] -= 1 << 33
    k, v, pos, ts = values
    batch["cache"] = oracle.qcache_rows(k, v, pos, ts, 4)
    _check(G, batch, values, slopes=([0.1, 0.0], [1e-9, 1e-10]))


def test_repeated_users(G):
    """The same user twice in a batch, and two users whose rows overlap (a shared prefix)."""
    batch, values = _batch(16, [(100, 3), (50, 2)], 8, 4, slack=0, order=[0, 1])
    for k in ("rows", "lens"):
        batch[k] = list(batch[k])
    batch["rows"] = [batch["rows"][0], batch["rows"][0], batch["rows"][0]]
    batch["lens"] = [100, 100, 40]
    batch["coff"] = np.array([0, 2, 4, 5])
    batch["tc"][:] = batch["tc"].max()
    o, _, _ = _check(G, batch, values)
    batch["qkv"][:, 2:4] = batch["qkv"][:, 0:2]
    o, _, _ = _check(G, batch, values)
    assert np.array_equal(o[0:2], o[2:4])


@pytest.mark.parametrize("bits", [8, 4])
def test_nan_and_infinity_stay_in_their_rows(G, bits):
    """A NaN head in a visible row makes that head's outputs NaN for that user's candidates; a
    NaN or infinite candidate only its own; rows of nobody reach nothing (see _batch's noise)."""
    users = [(40, 9), (40, 9)]
    batch, values = _batch(17, users, 4, bits)
    clean, _, _ = _score(G, batch["qkv"], batch["coff"], _dev(batch["cache"]), batch["rows"], batch["lens"], batch["tc"], 4, bits)
    for side in (0, 1):
        k, v, pos, ts = (x.copy() for x in values)
        (k if side == 0 else v)[batch["rows"][0] + 5, 1, 3] = np.inf
        rb = batch["cache"].copy()
        at = batch["rows"][0] + 5
        rb[at] = oracle.qcache_rows(k[at:at + 1], v[at:at + 1], pos[at:at + 1], ts[at:at + 1], bits)
        o, lse, code = _score(G, batch["qkv"], batch["coff"], _dev(rb), batch["rows"], batch["lens"], batch["tc"], 4, bits)
        assert code == 0
        assert np.isnan(o[:9, 1]).all() and np.array_equal(np.isnan(lse[:, :9]).any(1), [False, side == 0, False, False])
        keep = np.ones(o.shape[:2], bool)
        keep[:9, 1] = False
        assert np.array_equal(o[keep], clean[keep])
    qkv = batch["qkv"].copy()
    qkv[0, 2, 0, 5] = np.nan
    qkv[1, 4, 1, 6] = np.nan
    qkv[2, 6, 2, 7] = np.nan
    qkv[0, 8, 3, 7] = np.inf
    o, lse, code = _score(G, qkv, batch["coff"], _dev(batch["cache"]), batch["rows"], batch["lens"], batch["tc"], 4, bits)
    assert np.isnan(o[2, 0]).all() and np.isnan(o[4, 1]).all() and np.isnan(o[8, 3]).all()
    assert np.isnan(o[6, 2, 7]) and np.isnan(lse[:, 6]).sum() == 0
    keep = np.ones(o.shape[:2], bool)
    keep[[2, 4, 6, 8], [0, 1, 2, 3]] = False
    assert np.array_equal(o[keep], clean[keep])


# ------------------------------------------------------------------------------------------
# attention for many candidates: the kernel is chosen by the bounds of candidates and rows, so
# loose bounds (which the call allows) bring any batch to it
# ------------------------------------------------------------------------------------------

WIDE = dict(max_cand=1200, max_len=4096)
# lengths around the tile of 64 rows, candidates around the tile of 128
TILES = [(0, 130), (1, 1), (63, 127), (64, 128), (65, 129), (0, 0), (128, 0), (129, 300), (480, 41), (300, 257), (0, 1)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H", [1, 3, 8, 17])
def test_many_candidates(G, bits, H):
    _check(G, *_batch(30 + H, TILES, H, bits, tc_spread=5000), extra=3, **WIDE)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("users", [SMALL, LARGE], ids=["small", "large"])
def test_few_candidates_within_loose_bounds(G, bits, users):
    _check(G, *_batch(40, users, 5, bits, tc_spread=5000), extra=1, lse=False, **WIDE)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("m", [40, 41])
def test_both_sides_of_the_choice(G, bits, m):
    _check(G, *_batch(41, [(480, m)] * 60, 2, bits))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("users,H,bounds", [([(5000, 130)], 2, dict(max_cand=600)), ([(3000, 70), (0, 50), (700, 200)], 1, dict(max_cand=900)),
                                            ([(4097, 45)] * 3, 3, dict(max_cand=128))])
def test_many_candidates_in_ranges(G, bits, users, H, bounds):
    batch, values = _batch(42, users, H, bits)
    assert G.attn_qcached_workspace_size(len(users), len(batch["tc"]), H, 64, bounds["max_cand"], max(n for n, _ in users)) > 0
    _check(G, batch, values, extra=2, **bounds)


def test_more_items_than_blocks(G):
    """Every block walks over several items of unequal length, empty ones among them."""
    r = np.random.default_rng(43)
    users = [(int(r.integers(0, 200)), int(r.integers(0, 90))) for _ in range(150)]
    for bits in (8, 4):
        _check(G, *_batch(43, users, 4, bits), max_cand=128, max_len=1000)


@pytest.mark.parametrize("bits", [8, 4])
def test_small_caches_and_loose_bounds(G, bits):
    """Caches and candidate arrays shorter than a tile, and bounds far beyond what is there."""
    for users in ([(1, 50)], [(0, 41), (3, 2)], [(40, 3)]):
        for kw in (WIDE, dict(max_len=1 << 30), dict(max_cand=5000, max_len=100000)):
            _check(G, *_batch(53, users, 2, bits, slack=0), **kw)


def test_short_items_in_a_row(G):
    """Blocks walk over a dozen items each of no tile, one or two, and few or many candidates, whose
    roles' warps take different time."""
    r = np.random.default_rng(52)
    users = [(int(r.choice([0, 0, 1, 64, 64, 65, 150])), int(r.choice([1, 20, 33, 70, 100]))) for _ in range(700)]
    for bits in (8, 4):
        batch, values = _batch(52, users, 5, bits)
        first = _check(G, batch, values, max_cand=128, max_len=300)
        for _ in range(20):
            b = dict(batch)
            again = _score(G, b["qkv"], b["coff"], _dev(b["cache"]), b["rows"], b["lens"], b["tc"], 5, bits, max_cand=128, max_len=300)
            assert again[2] == 0 and np.array_equal(again[0], first[0]) and np.array_equal(again[1], first[1])


@pytest.mark.parametrize("bits", [8, 4])
def test_unequal_magnitudes_of_many_candidates(G, bits):
    """As test_unequal_magnitudes: the most recent tile is far from the maximum, in either direction."""
    batch, values = _batch(44, [(200, 60), (333, 130), (70, 3)], 4, bits, spread=10.0, qscale=1e-3)
    _check(G, batch, values, **WIDE)
    batch, values = _batch(45, [(200, 60), (333, 130), (70, 3)], 4, bits, qscale=60.0)
    batch["qkv"][1, ::3] *= 8.0
    batch["qkv"][1, 1::3] *= -8.0
    _check(G, batch, values, **WIDE)


@pytest.mark.parametrize("bits", [8, 4])
def test_small_values_outweigh_large_ones(G, bits):
    """Rows whose value scale is 2^-20 of the largest hold all the weight: they keep their bits."""
    H = 2
    batch, _ = _batch(46, [(150, 50)], H, bits, qscale=0.25)
    r, R = np.random.default_rng(46), len(batch["cache"])
    k, v = _kv(r, R, H), _kv(r, R, H)
    pos, ts = np.zeros(R, np.int64), np.zeros(R, np.int64)
    at = int(batch["rows"][0])
    pos[at:at + 150], ts[at:at + 150] = np.arange(1, 151), batch["tc"][0] - 9
    v[at:at + 150] *= np.float32(2.0 ** -20)
    v[at + 20] *= np.float32(2.0 ** 20)
    pos[at + 20] = 0
    batch["qkv"][2] *= np.float32(2.0 ** -20)
    batch["cache"] = oracle.qcache_rows(k, v, pos, ts, bits)
    for kw in (WIDE, {}):
        # the large row is left a weight below 2^-80 by its position
        _check(G, batch, (oracle.qcache_values(k, bits), oracle.qcache_values(v, bits), pos, ts), slopes=([0.5, 1.0], [0.0, 0.0]), **kw)


def test_extreme_magnitudes_of_many_candidates(G):
    """As test_extreme_magnitudes_of_q, with a zero and a tiny candidate among the others."""
    for up in (100, -100):
        for bits in (8, 4):
            batch, _ = _batch(47, [(77, 60)], 2, bits)
            r, n, R = np.random.default_rng(1), 77, len(batch["cache"])
            k, v = _kv(r, R, 2) * np.float32(2.0 ** -up), _kv(r, R, 2)
            pos, ts = np.zeros(R, np.int64), np.zeros(R, np.int64)
            s = slice(batch["rows"][0], batch["rows"][0] + n)
            pos[s], ts[s] = np.arange(1, n + 1), batch["tc"][0] - 5
            batch["cache"] = oracle.qcache_rows(k, v, pos, ts, bits)
            batch["qkv"][0] *= np.float32(2.0 ** up)
            batch["qkv"][0, 1] = 0.0
            batch["qkv"][0, 2] *= np.float32(2.0 ** -12)
            batch["qkv"][0, 3] *= np.float32(2.0 ** -80 if up > 0 else 2.0 ** -20)
            batch["qkv"][1] *= np.float32(2.0 ** -up)
            _check(G, batch, (oracle.qcache_values(k, bits), oracle.qcache_values(v, bits), pos, ts), **WIDE)
    batch, values = _batch(48, [(77, 60)], 2, 4)
    batch["qkv"][0] = 0.0  # every score is the bias, a user's keys are zero as well
    _check(G, batch, values, **WIDE)


@pytest.mark.parametrize("kw", [WIDE, {}], ids=["wide", "exact"])
def test_scores_beyond_floats_whole_numbers(G, kw):
    """Slopes that take every cached score to -1e9 and below, where neighbouring floats are 64 and
    more apart: the candidates' own scores hold all the weight, and nothing overflows."""
    for slopes in (([0.1, 0.0], [1.0, 30.0]), ([1e7, 1e8], [0.0, 0.0])):
        batch, values = _batch(49, [(300, 50), (64, 3)], 2, 4, qscale=8.0)
        k, v, pos, ts = values
        ts[ts > 0] -= 1 << 30
        batch["cache"] = oracle.qcache_rows(k, v, pos, ts, 4)
        o, _, _ = _check(G, batch, values, slopes=slopes, **kw)
        assert np.array_equal(o, batch["qkv"][2].astype(np.float64))


@pytest.mark.parametrize("bits", [8, 4])
def test_nan_and_infinity_stay_in_their_rows_of_many_candidates(G, bits):
    batch, values = _batch(50, [(140, 60), (140, 60)], 4, bits)
    b = batch

    def run(cache, qkv):
        return _score(G, qkv, b["coff"], _dev(cache), b["rows"], b["lens"], b["tc"], 4, bits, **WIDE)

    clean, _, code = run(b["cache"], b["qkv"])
    assert code == 0 and np.isfinite(clean).all()
    for side in (0, 1):
        k, v, pos, ts = (x.copy() for x in values)
        at = b["rows"][0] + 70
        (k if side == 0 else v)[at, 1, 3] = np.nan
        rb = b["cache"].copy()
        rb[at] = oracle.qcache_rows(k[at:at + 1], v[at:at + 1], pos[at:at + 1], ts[at:at + 1], bits)
        o, lse, code = run(rb, b["qkv"])
        assert code == 0
        assert np.isnan(o[:60, 1]).all() and np.array_equal(np.isnan(lse[:, :60]).any(1), [False, side == 0, False, False])
        keep = np.ones(o.shape[:2], bool)
        keep[:60, 1] = False
        assert np.array_equal(o[keep], clean[keep])
    qkv = b["qkv"].copy()
    qkv[0, 2, 0, 5] = np.nan
    qkv[1, 4, 1, 6] = np.nan
    qkv[2, 6, 2, 7] = np.nan
    qkv[0, 8, 3, 7] = np.inf
    qkv[0, 61, 3, 7] = -np.inf
    o, lse, code = run(b["cache"], qkv)
    assert code == 0
    assert np.isnan(o[2, 0]).all() and np.isnan(o[4, 1]).all() and np.isnan(o[8, 3]).all() and np.isnan(o[61, 3]).all()
    assert np.isnan(o[6, 2, 7]) and np.isnan(lse[:, 6]).sum() == 0
    keep = np.ones(o.shape[:2], bool)
    keep[[2, 4, 6, 8, 61], [0, 1, 2, 3, 3]] = False
    assert np.array_equal(o[keep], clean[keep])


def test_errors_of_many_candidates(G):
    batch, values = _batch(51, [(140, 50), (133, 60), (70, 50)], 2, 4, order=[0, 1, 2])
    b = {k: (list(v) if k in ("rows", "lens") else v) for k, v in batch.items()}
    cache = _dev(b["cache"])
    R = len(b["cache"])

    def run(max_cand=1200, max_len=4096, **kw):
        a = {**b, **kw}
        return _score(G, a["qkv"], a["coff"], cache, a["rows"], a["lens"], a["tc"], 2, 4, max_cand=max_cand, max_len=max_len)

    clean, _, code = run()
    assert code == 0
    left = np.ones(160, bool)
    left[50:110] = False
    for kw in (dict(rows=[b["rows"][0], R - 5, b["rows"][2]]), dict(rows=[b["rows"][0], -1, b["rows"][2]]),
               dict(lens=[140, -1, 70])):
        o, lse, code = run(**kw)
        assert code == G.DERR["LAYOUT"]
        assert np.isnan(o[50:110]).all() and np.array_equal(o[left], clean[left])
    assert run(coff=np.array([0, 50, 110, 170]))[2] == G.DERR["LAYOUT"]
    o, _, code = run(max_cand=55, max_len=8192)  # the second user's last five are left out
    assert code == G.DERR["LAYOUT"] and np.isnan(o[105:110]).all()
    assert np.array_equal(np.delete(o, range(105, 110), 0), np.delete(clean, range(105, 110), 0))
    assert run(max_len=139)[2] == G.DERR["LAYOUT"]
    tc = b["tc"].copy()
    tc[70] -= 1 << 30
    o, _, code = run(tc=tc)
    assert code == G.DERR["TS_ORDER"] and np.array_equal(o[:50], clean[:50])
    k, v, pos, ts = values
    pos[b["rows"][2] + 3] = 200
    cache = _dev(oracle.qcache_rows(k, v, pos, ts, 4))
    o, _, code = run()
    assert code == G.DERR["POS_RANGE"] and np.array_equal(o[:110], clean[:110])


def test_attention_layout_and_order_errors(G):
    batch, values = _batch(18, [(40, 2), (33, 3), (20, 2)], 2, 4, order=[0, 1, 2])
    b = {k: (list(v) if k in ("rows", "lens") else v) for k, v in batch.items()}
    cache = _dev(b["cache"])
    R = len(b["cache"])

    def run(**kw):
        a = {**b, **kw}
        return _score(G, a["qkv"], a["coff"], cache, a["rows"], a["lens"], a["tc"], 2, 4,
                      max_cand=a.get("max_cand"), max_len=a.get("max_len"))

    clean, _, code = run()
    assert code == 0
    left = np.ones(7, bool)
    left[2:5] = False
    for kw in (dict(rows=[b["rows"][0], R - 5, b["rows"][2]]), dict(rows=[b["rows"][0], -1, b["rows"][2]]),
               dict(lens=[40, -1, 20])):
        o, lse, code = run(**kw)
        assert code == G.DERR["LAYOUT"]
        assert np.isnan(o[2:5]).all() and np.array_equal(o[left], clean[left])
    o, _, code = run(max_cand=2)  # the third candidate of the second user is left out
    assert code == G.DERR["LAYOUT"] and np.isnan(o[4]).all() and np.array_equal(np.delete(o, 4, 0), np.delete(clean, 4, 0))
    assert run(max_len=39)[2] == G.DERR["LAYOUT"]
    assert run(coff=np.array([0, 2, 5, 9]))[2] == G.DERR["LAYOUT"]
    tc = b["tc"].copy()
    tc[3] -= 1 << 30
    o, _, code = run(tc=tc)
    assert code == G.DERR["TS_ORDER"] and np.array_equal(o[:2], clean[:2])


def test_equal_to_cached_attention_over_the_read_back(G):
    """What the quantised attention gives is genrank_attn_fwd_cached over the rows read back, to
    the rounding of that kernel's bf16 softmax weights (2^-8 of each, and of the output)."""
    H, bits = 8, 4
    batch, values = _batch(19, [(480, 40), (17, 3), (0, 2), (129, 20)], H, bits, slack=0, order=[0, 1, 2, 3])
    o, lse, code = _score(G, batch["qkv"], batch["coff"], _dev(batch["cache"]), batch["rows"], batch["lens"], batch["tc"], H, bits)
    assert code == 0
    d, C, Th = H * 64, len(batch["tc"]), sum(batch["lens"])
    hoff = _dev(np.concatenate([[0], np.cumsum(batch["lens"])]), torch.int32)
    kv = torch.empty(Th, 2 * d, dtype=torch.bfloat16, device="cuda")
    pos = torch.empty(Th, dtype=torch.int32, device="cuda")
    ts = torch.empty(Th, dtype=torch.int64, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    G.qcache_read(hoff, None, _dev(batch["cache"]), _dev(batch["rows"], torch.int64), kv, kv[:, d:], 2 * d, H, 64, pos, ts,
                  G.QCACHE_INT4, err)
    x = _dev(batch["qkv"].transpose(1, 0, 2, 3).reshape(C, 3 * d), torch.bfloat16)
    ws = torch.empty(G.attn_cached_workspace_size(4, C, Th, H, 64, 40), dtype=torch.uint8, device="cuda")
    oc = torch.empty(C, d, dtype=torch.bfloat16, device="cuda")
    lc = torch.empty(H, C, dtype=torch.float32, device="cuda")
    sp, st = G.alibi_slopes(H)
    G.attn_fwd_cached(_dev(batch["coff"], torch.int32), 40, x, x[:, d:], x[:, 2 * d:], 3 * d, hoff, kv, kv[:, d:], 2 * d,
                      pos, ts, _dev(batch["tc"], torch.int64), H, 64, sp, st, 0.125, oc, d, lc, ws, err, C=C, Th=Th)
    assert G.check_error(err) == 0
    qkv = batch["qkv"].astype(np.float64)
    _, _, A, _ = oracle.attention_fwd_qcached(*qkv, batch["coff"], values[0], values[1], batch["rows"], batch["lens"],
                                              values[2], values[3], batch["tc"], sp, st, 0.125)
    oc = oc.double().cpu().numpy().reshape(C, H, 64)
    assert np.all(np.abs(o - oc) <= 2.0 ** -7 * np.abs(oc) + 2.0 ** -7 * A)
    assert np.max(np.abs(lse - lc.double().cpu().numpy())) <= 1e-3


# ------------------------------------------------------------------------------------------
# together, and under streams and graphs
# ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("bits", [8, 4])
def test_a_server_s_run(G, bits):
    """Histories written from a fused projection, tokens appended one at a time, scored after
    each: as if every key and value had been quantised at once."""
    r = np.random.default_rng(21)
    B, H, m, room = 5, 8, 3, 50
    d, fmt = H * 64, _fmt(G, bits)
    n = np.array([0, 3, 31, 32, 40])
    k, v = _kv(r, B * room, H).reshape(B, room, H, 64), _kv(r, B * room, H).reshape(B, room, H, 64)
    ts = 1_700_000_000 + np.cumsum(r.integers(0, 900, (B, room)), 1)
    first = np.arange(B) * room
    cache = torch.full((B * room, G.qcache_row_bytes(H, 64, fmt)), 0xFF, dtype=torch.uint8, device="cuda")
    # the fused projection of the scoring layout: each user's history, then its candidates
    seq = np.concatenate([[0], np.cumsum(n + m)])
    qkv = torch.zeros(int(seq[-1]), 3 * d, dtype=torch.bfloat16, device="cuda")
    pos0, ts0 = np.zeros(int(seq[-1])), np.zeros(int(seq[-1]))
    for u in range(B):
        s = slice(int(seq[u]), int(seq[u]) + int(n[u]))
        qkv[s, d:2 * d] = _dev(k[u, :n[u]].reshape(-1, d))
        qkv[s, 2 * d:] = _dev(v[u, :n[u]].reshape(-1, d))
        pos0[s], ts0[s] = np.arange(1, n[u] + 1), ts[u, :n[u]]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    G.qcache_append(_dev(seq, torch.int32), _dev(n, torch.int32), qkv[:, d:], qkv[:, 2 * d:], 3 * d, H, 64,
                    _dev(pos0, torch.int32), _dev(ts0, torch.int64), cache, _dev(first, torch.int64), fmt, err)
    values = (oracle.qcache_values(k.reshape(-1, H, 64), bits), oracle.qcache_values(v.reshape(-1, H, 64), bits),
              np.tile(np.arange(1, room + 1), B), ts.reshape(-1))
    one = _dev(np.arange(B + 1), torch.int32)
    for step in range(4):
        at = np.arange(B), n
        G.qcache_append(one, None, _dev(k[at].reshape(B, d), torch.bfloat16), _dev(v[at].reshape(B, d), torch.bfloat16), d,
                        H, 64, _dev(n + 1, torch.int32), _dev(ts[at], torch.int64), cache, _dev(first + n, torch.int64), fmt, err)
        n = n + 1
        q = np.stack([_bf16(r.standard_normal((B * m, H, 64))) for _ in range(3)])
        tc = np.repeat(ts[np.arange(B), n - 1] + 60, m)
        _compare(G, q, np.arange(B + 1) * m, cache, first, n.tolist(), tc, H, bits, values)
    assert G.check_error(err) == 0
    untouched = np.concatenate([np.arange(first[u] + n[u], first[u] + room) for u in range(B)])
    assert (cache[_dev(untouched)] == 0xFF).all()


def test_streams_and_graphs(G):
    """Calls on a side stream; captured graphs (joined and direct ones, few candidates and many) replayed in turn on
    changed inputs, bit for bit the eager results."""
    cases = [_batch(22, [(700, 2)], 8, 4), _batch(23, [(50, 3)] * 200, 8, 8), _batch(24, [(3000, 60)] * 2, 8, 4),
             _batch(25, [(500, 50)] * 50, 8, 8)]
    H, d, fmts = 8, 512, [G.QCACHE_INT4, G.QCACHE_INT8] * 2
    sp, st = G.alibi_slopes(H)
    calls = []
    for (b, _), fmt in zip(cases, fmts):
        C = len(b["tc"])
        x = _dev(b["qkv"].transpose(1, 0, 2, 3).reshape(C, 3 * d), torch.bfloat16)
        mc, ml = int(np.diff(b["coff"]).max()), int(max(b["lens"]))
        ws = torch.empty(max(16, G.attn_qcached_workspace_size(len(b["rows"]), C, H, 64, mc, ml)), dtype=torch.uint8, device="cuda")
        o = torch.zeros(C, d, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(H, C, dtype=torch.float32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        args = (_dev(b["coff"], torch.int32), mc, x, x[:, d:], x[:, 2 * d:], 3 * d, _dev(b["cache"]), _dev(b["rows"], torch.int64),
                _dev(b["lens"], torch.int32), ml, _dev(b["tc"], torch.int64), H, 64, sp, st, 0.125, o, d, lse, ws, fmt, err)
        calls.append((x, o, lse, err, args))
    assert G.attn_qcached_workspace_size(1, 2, H, 64, 2, 700) > 0
    graphs = []
    side = torch.cuda.Stream()
    for _, _, _, _, args in calls:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            G.attn_fwd_qcached(*args)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            G.attn_fwd_qcached(*args)
        graphs.append(g)
    for rep in range(3):
        for x, *_ in calls:
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(rep)))
        want = []
        for _, o, lse, _, args in calls:
            G.attn_fwd_qcached(*args)
            want.append((o.clone(), lse.clone()))
            o.zero_()
        for g in graphs:
            g.replay()
        for (_, o, lse, err, _), (wo, wl) in zip(calls, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)
            assert G.check_error(err) == 0


def test_python_refusals_on_the_gpu(G):
    H, d = 2, 128
    cache = torch.zeros(8, G.qcache_row_bytes(H, 64, G.QCACHE_INT8), dtype=torch.uint8, device="cuda")
    k = torch.zeros(4, d, dtype=torch.bfloat16, device="cuda")
    off, rows = _dev([0, 4], torch.int32), _dev([0], torch.int64)
    pos, ts, err = _dev(range(4), torch.int32), _dev(range(4), torch.int64), _dev([0], torch.int32)

    def append(**kw):
        a = dict(off=off, k=k, v=k, stride=d, pos=pos, ts=ts, cache=cache, rows=rows, T=None)
        a.update(kw)
        G.qcache_append(a["off"], None, a["k"], a["v"], a["stride"], H, 64, a["pos"], a["ts"], a["cache"], a["rows"],
                        G.QCACHE_INT8, err, T=a["T"])

    append()
    for kw in (dict(off=off.long()), dict(rows=rows.int()), dict(v=k.float()), dict(pos=pos.long()), dict(ts=ts.int()),
               dict(cache=cache[:, :-16]), dict(pos=pos.cpu()), dict(off=off[:1]), dict(stride=2 * d), dict(T=5),
               dict(k=k.half(), v=k.half()), dict(k=k[:, 4:])):
        with pytest.raises(G.GenRankError):
            append(**kw)
    assert G.check_error(err) == 0


# ------------------------------------------------------------------------------------------
# long token arrays: a warp walks several rows
# ------------------------------------------------------------------------------------------

def _long_batch(seed, T, first, H, bits):
    """Segments of every length from offset `first` on, some rows of each written, rows of nobody
    behind the last; tokens out of a pool of 300 and the pool's cache rows."""
    r = np.random.default_rng(seed)
    seg = []
    while first + sum(seg) < T - 2100:
        seg.append(int(r.choice([0, 0, 1, 2, 7, 64, 300, 2000])))
    seg = np.array(seg)
    length = np.array([int(r.integers(0, s + 1)) if r.random() < 0.5 else s for s in seg])
    off = first + np.concatenate([[0], np.cumsum(seg)])
    k, v = _kv(r, 300, H, 6.0), _kv(r, 300, H, 6.0)
    pos, ts = r.integers(1, 1000, 300), r.integers(0, 1 << 40, 300)
    at = np.concatenate([[0], np.cumsum(length + r.integers(0, 3, len(seg)))]) + 1
    of = np.concatenate([np.arange(o, o + n) for o, n in zip(off, length)])  # token rows copied
    to = np.concatenate([np.arange(a, a + n) for a, n in zip(at, length)])   # and their cache rows
    return dict(off=off, length=length, k=k, v=v, pos=pos, ts=ts, at=at, of=of, to=to, token=r.integers(0, 300, T),
                pool=oracle.qcache_rows(k, v, pos, ts, bits))


LONG = [(1, 200000, 5), (8, 40000, 1), (9, 30000, 481), (2, 20000, 0)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H,T,first", LONG)
def test_append_long_arrays(G, bits, H, T, first):
    b = _long_batch(T + first, T, first, H, bits)
    i = b["token"]
    R = int(b["at"][-1]) + 2
    cache, code = _append(G, b["k"][i], b["v"][i], b["pos"][i], b["ts"][i], b["off"], b["length"], b["at"][:-1], R, bits)
    assert code == 0
    want = np.full((R, cache.shape[1]), 0x5A, np.uint8)
    want[b["to"]] = b["pool"][i[b["of"]]]
    assert np.array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H,T,first", LONG)
def test_read_long_arrays(G, bits, H, T, first):
    b = _long_batch(T + first, T, first, H, bits)
    r = np.random.default_rng(first)
    at = r.integers(0, 5000 - 2000, len(b["length"]))  # rows in any order, shared by users
    token = r.integers(0, 300, 5000)
    out = torch.full((2, T, H * 64), -7.0, dtype=torch.bfloat16, device="cuda")
    po = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    to = torch.full((T,), -7, dtype=torch.int64, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    G.qcache_read(_dev(b["off"], torch.int32), _dev(b["length"], torch.int32), _dev(b["pool"][token]), _dev(at, torch.int64),
                  out[0], out[1], H * 64, H, 64, po, to, _fmt(G, bits), err)
    assert G.check_error(err) == 0
    src = token[np.concatenate([np.arange(a, a + n) for a, n in zip(at, b["length"])])]
    for side, x in enumerate((b["k"], b["v"])):
        want = np.full((T, H * 64), -7.0, np.float32)
        want[b["of"]] = oracle.qcache_values(x, bits).reshape(300, -1)[src]
        assert np.array_equal(out[side].float().cpu().numpy(), want)
    wp, wt = np.full(T, -7), np.full(T, -7)
    wp[b["of"]], wt[b["of"]] = b["pos"][src], b["ts"][src]
    assert np.array_equal(po.cpu().numpy(), wp) and np.array_equal(to.cpu().numpy(), wt)


def test_append_never_writes_a_row_twice(G):
    """Users whose first rows do not ascend: whatever is left out, those written are whole and apart
    from one another, a user in order with all others is written, and the call is flagged."""
    r = np.random.default_rng(70)
    n_tok, H, bits = 400, 1, 4
    k, v = _kv(r, n_tok, H), _kv(r, n_tok, H)
    pos, ts = np.arange(n_tok), np.arange(n_tok)
    rows_of = oracle.qcache_rows(k, v, pos, ts, bits)
    shapes = [([0, 50, 3], [5, 1, 5]), ([0, 50, 3, 4], [5, 1, 1, 1]), ([3, 50, 0, 1, 2], [5, 1, 1, 1, 9]),
              ([90, 5, 5, 5, 7], [1, 2, 2, 0, 0])]
    for _ in range(60):
        B = int(r.integers(2, 40))
        n = r.integers(0, 9, B)
        at = np.concatenate([[0], np.cumsum(n)])[:-1] + 3
        for _ in range(int(r.integers(0, 4))):  # some moved, or swapped
            i, j = r.integers(0, B, 2)
            at[i] = at[j] if r.random() < 0.5 else int(r.integers(-2, 420))
        shapes.append((at, n))
    for at, n in shapes:
        at, n = np.asarray(at, np.int64), np.asarray(n)
        off = np.concatenate([[0], np.cumsum(n)])
        T, R = int(off[-1]) + 1, 410
        cache, code = _append(G, k[:T], v[:T], pos[:T], ts[:T], off, None, at, R, bits)
        got = cache.cpu().numpy()
        end = at + n
        fits = (at >= 0) & (end <= R)
        good = bool(fits.all() and (end[:-1] <= at[1:]).all())
        assert (code == 0) == good and code in (0, G.DERR["LAYOUT"])
        written = np.zeros(R, int)
        for u in range(len(n)):
            in_order = fits[u] and (end[:u] <= at[u]).all() and (at[u + 1:] >= end[u]).all() and (at[:u] <= at[u]).all()
            whole = bool(fits[u]) and np.array_equal(got[at[u]:end[u]], rows_of[off[u]:off[u + 1]])
            assert whole or not in_order
            if whole:
                written[at[u]:end[u]] += 1
        assert written.max(initial=0) <= 1
        assert np.array_equal(written > 0, (got != 0x5A).any(-1))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("m,kw", [(8, {}), (8, WIDE), (40, WIDE)], ids=["few", "many", "40"])
def test_a_candidate_beside_an_outlier(G, bits, m, kw):
    """One candidate's q a factor up to 2^60 above the others': each keeps its own precision, and
    is bit for bit what it is alone (under the same bounds)."""
    batch, values = _batch(60, [(480, m)], 3, bits)
    few = not kw
    kw = dict(kw or dict(max_cand=m, max_len=480))
    plain = batch["qkv"]
    for up in (12, 17, 20, 24, 60) if few else (12, 17, 20, 24):
        batch["qkv"] = plain.copy()
        batch["qkv"][0, 1] *= np.float32(2.0 ** up)
        o, lse, _ = _check(G, batch, values, **kw)
        for c in (0, 1, 5, m - 1):
            one, ls, code = _score(G, batch["qkv"][:, c:c + 1], [0, 1], _dev(batch["cache"]), batch["rows"], batch["lens"],
                                   batch["tc"][c:c + 1], 3, bits, **kw)
            assert code == 0 and np.array_equal(one[0], o[c]) and np.array_equal(ls[:, 0], lse[:, c])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("kw", [{}, WIDE], ids=["few", "many"])
def test_scores_far_beyond_whole_numbers(G, bits, kw):
    """Scores q.k from 2^26 to 2^80, between which floats are many log2 units apart: the largest holds
    the weight, alone or with those equal to it, whichever tile it is in."""
    batch, values = _batch(66, [(300, 8), (65, 3), (1, 2)], 3, bits)
    plain = batch["qkv"]
    for up in (26, 29, 33, 40, 60, 80):
        batch["qkv"] = plain.copy()
        batch["qkv"][0] *= np.float32(2.0 ** up)
        batch["qkv"][0, 5] *= np.float32(2.0 ** -up)  # an ordinary one among them
        o, lse, _ = _check(G, batch, values, **kw)
        k, v = (np.asarray(x, np.float64) for x in values[:2])
        qkv = batch["qkv"].astype(np.float64)
        for c in (0, 1, 2, 3, 4, 8, 9):
            u = 0 if c < 8 else 1
            s = slice(batch["rows"][u], batch["rows"][u] + batch["lens"][u])
            for h in range(3):
                x = np.concatenate([k[s, h] @ qkv[0, c, h], [qkv[1, c, h] @ qkv[0, c, h]]])
                i, second = int(x.argmax()), np.sort(x)[-2]
                mag = np.abs(qkv[0, c, h]) @ np.abs(np.concatenate([k[s, h], qkv[1, c:c + 1, h]])).max(0)
                if x[i] - second > 2.0 ** -17 * mag:  # apart by more than fp32 sums may be off
                    one = v[s, h][i] if i < batch["lens"][u] else qkv[2, c, h]
                    assert np.array_equal(o[c, h], one), (up, c, h)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("kw", [WIDE, {}], ids=["many", "few"])
@pytest.mark.parametrize("scale,slope", [(2.0 ** -100, 0.0), (2.0 ** -140, 0.02), (2.0 ** -60, 1e-30), (2.0 ** -100, 3e38),
                                         (0.125, 3e38), (0.125, 2e30), (2.0 ** 40, 0.5)])
def test_scales_and_slopes_of_any_size(G, bits, kw, scale, slope):
    """Scores that vanish, biases beyond fp32: histories that end inside a tile of either form."""
    H, users = 2, [(70, 5), (33, 3), (1, 2)]
    batch, values = _batch(62, users, H, bits)
    k, v, pos, ts = values
    last = batch["rows"][0] + 69
    ts[last] = batch["tc"][0]  # no time between the candidates and this row
    batch["cache"] = oracle.qcache_rows(k, v, pos, ts, bits)
    if scale > 1.0:
        batch["qkv"][0] *= np.float32(2.0 ** -40)
    C, d = 10, H * 64
    x = _dev(batch["qkv"].transpose(1, 0, 2, 3).reshape(C, 3 * d), torch.bfloat16)
    mc, ml = kw.get("max_cand", 5), kw.get("max_len", 70)
    ws = torch.empty(max(16, G.attn_qcached_workspace_size(3, C, H, 64, mc, ml)), dtype=torch.uint8, device="cuda")
    o = torch.empty(C, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(H, C, dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for sp, st in (([slope, 0.0], [0.0, 0.0]), ([0.0, 0.0], [slope, slope / 1024])):
        sp, st = ([float(np.float32(s)) for s in z] for z in (sp, st))
        G.attn_fwd_qcached(_dev(batch["coff"], torch.int32), mc, x, x[:, d:], x[:, 2 * d:], 3 * d, _dev(batch["cache"]),
                           _dev(batch["rows"], torch.int64), _dev(batch["lens"], torch.int32), ml, _dev(batch["tc"], torch.int64),
                           H, 64, sp, st, scale, o, d, lse, ws, _fmt(G, bits), err)
        assert G.check_error(err) == 0
        want, wl, A, S = oracle.attention_fwd_qcached(*batch["qkv"].astype(np.float64), batch["coff"], k, v, batch["rows"],
                                                      batch["lens"], pos, ts, batch["tc"], sp, st, scale)
        e = 2.0 ** -18 * S + 2.0 ** -19
        got = o.double().cpu().numpy().reshape(C, H, 64)
        tol = 2.0 ** -8 * np.abs(want) + A * (2.0 ** -11 + 2 * e.T[:, :, None]) + 70 * 2.0 ** -30 * np.abs(v).max()
        assert np.all(np.abs(got - want) <= tol), np.nanmax(np.abs(got - want) / tol)
        assert np.all(np.abs(lse.double().cpu().numpy() - wl) <= e + 2.0 ** -22 * np.abs(wl))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("users,kw", [([(200, 8), (90, 3)], {}), ([(200, 8), (90, 3)], WIDE), ([(3000, 5)], {}),
                                      ([(3000, 60)], dict(max_cand=900))], ids=["few", "many", "few-ranges", "many-ranges"])
def test_candidates_far_apart_in_time(G, bits, users, kw):
    """A week between a user's candidates, the first one the latest, and slopes by which the history
    matters to the early ones: no score is the difference of two large numbers, and the order of the
    candidates does not matter.  A bias of x nats weighs e^-x, so that only those up to 64 count in
    the LSE, each rounded to 2^-22 of itself."""
    H = 2
    batch, values = _batch(63, users, H, bits)
    k, v, pos, ts = values
    c0 = np.array(batch["coff"])
    slopes = ([0.0, 0.0], [1.0 / 16, 1.0 / 64])
    for u, (n, m) in enumerate(users):
        t0 = 1_700_000_000
        ts[batch["rows"][u]:batch["rows"][u] + n] = t0 - 3 * np.arange(n)[::-1] - 5
        tc = t0 + np.arange(m) * 7
        tc[0] = t0 + 7 * 86400
        tc[m // 2] = t0 + 3 * 86400
        batch["tc"][c0[u]:c0[u + 1]] = tc
    batch["cache"] = oracle.qcache_rows(k, v, pos, ts, bits)
    o, lse, _ = _check(G, batch, values, slopes=slopes, **kw)
    want, wl, A, S = oracle.attention_fwd_qcached(*batch["qkv"].astype(np.float64), batch["coff"], k, v, batch["rows"],
                                                  batch["lens"], pos, ts, batch["tc"], *slopes, 0.125)
    err = np.abs(lse - wl)
    tol = 2.0 ** -18 * S + 2.0 ** -19 + 2.0 ** -22 * (np.abs(wl) + 64)
    assert np.all(err <= tol), np.max(err / tol)
    turn = np.concatenate([np.arange(c0[u], c0[u + 1])[::-1] for u in range(len(users))])
    b = dict(batch, qkv=batch["qkv"][:, turn], tc=batch["tc"][turn])
    back, lback, _ = _check(G, b, values, slopes=slopes, **kw)
    assert np.array_equal(back, o[turn]) and np.array_equal(lback, lse[:, turn])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("kw", [{}, WIDE], ids=["few", "many"])
def test_value_scales_far_below_the_largest(G, bits, kw):
    """One row of large values and no weight before two of small ones.  Few candidates: a weight times
    its value scale enters the product in fp16 under 2^11 over a power of two at most twice the
    largest scale, where half a step of the smallest numbers is 2^-25, so that a row is off by 2^-35
    of the largest value at most.  Many: value scales down to 2^-25 (8 bits: 2^-30) of the largest
    are exact; heads' scales differ by up to a factor of 6 here."""
    H, n = 4, 3
    for down in (15, 20, 28) if not kw else (15, 20, 22 if bits == 4 else 27):
        batch, _ = _batch(64, [(n, 8)], H, bits, qscale=0.5)
        r, R = np.random.default_rng(64), len(batch["cache"])
        k, v = _kv(r, R, H), _kv(r, R, H)
        pos, ts = np.zeros(R, np.int64), np.zeros(R, np.int64)
        at = int(batch["rows"][0])
        pos[at + 1:at + n], ts[at:at + n] = n + 1, batch["tc"][0] - 9
        v[at + 1:at + n] *= np.float32(2.0 ** -down)
        batch["qkv"][2] *= np.float32(2.0 ** -down)
        batch["cache"] = oracle.qcache_rows(k, v, pos, ts, bits)
        slopes = ([40.0] * H, [0.0] * H)  # 160 nats for the first row, none for the others
        o, _, code = _score(G, batch["qkv"], batch["coff"], _dev(batch["cache"]), batch["rows"], batch["lens"], batch["tc"], H, bits,
                            slopes=slopes, **kw)
        assert code == 0
        want, _, A, S = oracle.attention_fwd_qcached(*batch["qkv"].astype(np.float64), batch["coff"], oracle.qcache_values(k, bits),
                                                     oracle.qcache_values(v, bits), batch["rows"], batch["lens"], pos, ts,
                                                     batch["tc"], *slopes, 0.125)
        e = (2.0 ** -18 * S + 2.0 ** -19).T[:, :, None]
        tol = 2.0 ** -8 * np.abs(want) + A * (2.0 ** -11 + 2 * e) + (0.0 if kw else (n - 1) * 2.0 ** -35 * np.abs(v[at]).max())
        assert np.all(np.abs(o - want) <= tol), (down, np.max(np.abs(o - want) / tol))


def test_slopes_changed_in_place(G):
    """Slopes given as tensors, changed between two calls: the second call sees the new ones."""
    batch, values = _batch(65, [(60, 2)], 2, 4)
    slopes = [[torch.tensor(0.5), torch.tensor(0.25)], [torch.tensor(0.0), torch.tensor(0.0)]]
    for x in (0.5, 0.01, 3.0):
        for t in slopes[0]:
            t.fill_(x)
        _check(G, batch, values, slopes=slopes)
