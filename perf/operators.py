"""Workloads of the quantised history cache: appending K/V rows to it, reading them back, and
scoring candidates against it.

A case is one call (append: the write and the read-back of the rows written).  ``own`` selects
the library's entry points; otherwise the same results come from elementary torch operations in
fp32.  ``exact`` computes them in float64 from the definitions.

The cache holds one row of bytes per token:
  [K codes: H x cb][V codes: H x cb][H x (K scale, V scale) bf16][zeros to 16 B]
  [ts int64, pos int32, 0 int32][zeros to an odd multiple of 16 B]
with cb = 64 (int8, a byte c + 128 per value) or 32 (int4, a nibble c + 8, low nibble first), and
a value c * scale per code.  The scale belongs to one token, head and side (K or V):
  int8: the smallest power of two s with max|x| <= 127 s (exponent in [-126, 121])
  int4: max|x| / 7 to five significant bits, halves up (in [2^-126, 36 * 2^120])
  c = sign(x) floor(|x| / s + 1/2), at most 127 or 7
"""
import math

import numpy as np
import torch

own = False

DH = 64
FMTS = {"int8": 0, "int4": 1}
SLACK = 5  # rows that a user owns in the cache beyond those in use, at most
T_REQ = 1_750_000_000


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # one new interaction of each of a request batch's users
        dict(name="append_token", kind="append", fmt="int4", src="bf16", B=64, L=1, ragged=False, H=8, shape_seed=1),
        # a stream's update: one interaction of each of many users, from fp32 projections
        dict(name="append_tokens_f32", kind="append", fmt="int8", src="f32", B=2048, L=1, ragged=False, H=8, shape_seed=2),
        # histories of the training workload's lengths, written in one call
        dict(name="append_ragged", kind="append", fmt="int8", src="bf16", B=512, L=480, ragged=True, H=8, shape_seed=3),
        # the four-layer scoring workload's histories, one layer
        dict(name="append_histories", kind="append", fmt="int4", src="bf16", B=1024, L=480, ragged=False, H=8, shape_seed=4),
        # one user's history read back, as when a cache is handed on or re-quantised
        dict(name="read_user", kind="read", fmt="int8", src="bf16", B=1, L=480, ragged=False, H=4, shape_seed=5),
        dict(name="read_ragged_f32", kind="read", fmt="int4", src="f32", B=256, L=2048, ragged=True, H=8, shape_seed=6),
        # one candidate of one user: the smallest scoring call
        dict(name="score_one", kind="score", fmt="int4", B=1, L=480, ragged=False, m=1, m_ragged=False, H=8, lse=True, shape_seed=7),
        # a token at a time over longer histories
        dict(name="score_single_tokens", kind="score", fmt="int4", B=256, L=4096, ragged=False, m=1, m_ragged=False, H=8, lse=False, shape_seed=8),
        # a few users' lifelong histories
        dict(name="score_lifelong", kind="score", fmt="int8", B=4, L=65536, ragged=False, m=8, m_ragged=False, H=8, lse=True, shape_seed=9),
        # a mixed request batch: odd head count, users without history or candidates
        dict(name="score_ragged", kind="score", fmt="int8", B=300, L=2000, ragged=True, m=33, m_ragged=True, H=5, lse=True, shape_seed=10),
        # the candidate sweep's largest point
        dict(name="score_sweep", kind="score", fmt="int8", B=64, L=480, ragged=False, m=1024, m_ragged=False, H=16, lse=False, shape_seed=11),
        # the four-layer scoring workload's candidates
        dict(name="score_batch", kind="score", fmt="int4", B=1024, L=480, ragged=False, m=256, m_ragged=False, H=8, lse=False, shape_seed=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    kind = rng.choice(("append", "read", "score", "score"))
    c = dict(kind=kind, fmt=rng.choice(("int8", "int4")), H=rng.choice((1, 2, 3, 4, 5, 8, 8, 11, 12, 16)),
             ragged=rng.random() < 0.6, shape_seed=rng.randrange(1 << 30))
    if kind == "score":
        c.update(m=_log_int(rng, 1, 1024), m_ragged=rng.random() < 0.5, lse=rng.random() < 0.5)
        c.update(B=_log_int(rng, 1, 1024), L=_log_int(rng, 1, 65536))
        # the padded score matrix of the plain form stays within the largest listed case's
        while c["B"] > 1 and (c["B"] * c["L"] * c["m"] * c["H"] > 1 << 30 or c["B"] * c["L"] * c["H"] > 8 << 20 or _cost(c) > 4e9):
            c["B"] = (c["B"] + 1) // 2
        while c["L"] > 1 and (c["L"] * c["m"] * c["H"] > 1 << 30 or _cost(c) > 4e9):
            c["L"] = (c["L"] + 1) // 2
    else:
        c.update(src=rng.choice(("bf16", "f32")), B=_log_int(rng, 1, 4096), L=_log_int(rng, 1, 4096))
        while c["B"] > 1 and c["B"] * c["L"] * c["H"] > 3 << 20:
            c["B"] = (c["B"] + 1) // 2
    return c


def _shape(c):
    """Host-side sizes of a case: rows held by each user, candidates of each user, and the users'
    first cache rows (in cache order for a write, in any order for a read)."""
    r = np.random.RandomState(c["shape_seed"] % (1 << 31))
    n = r.randint(0, c["L"] + 1, c["B"]) if c["ragged"] else np.full(c["B"], c["L"])
    if c["ragged"]:
        n[r.randint(0, c["B"])] = c["L"]
    m = np.zeros(c["B"], np.int64)
    if c["kind"] == "score":
        m = r.randint(0, c["m"] + 1, c["B"]) if c["m_ragged"] else np.full(c["B"], c["m"])
        if c["m_ragged"]:
            m[r.randint(0, c["B"])] = c["m"]
    slack = r.randint(0, SLACK + 1, c["B"])
    order = np.arange(c["B"]) if c["kind"] == "append" else r.permutation(c["B"])
    begin = np.zeros(c["B"], np.int64)
    begin[order] = np.concatenate([[0], np.cumsum((n + slack)[order])])[:-1]
    return dict(n=n.astype(np.int64), m=m.astype(np.int64), begin=begin, rows=int((n + slack).sum()))


def _layout(H, fmt):
    """(code bytes of a head, offset of the scales, offset of ts and pos, bytes of a row)."""
    cb = 64 if fmt == "int8" else 32
    scales = 2 * H * cb
    tail = (scales + 4 * H + 15) // 16 * 16
    row = tail + 16
    return cb, scales, tail, row + (0 if row // 16 % 2 else 16)


def work(case):
    sh = _shape(case)
    H, d = case["H"], case["H"] * DH
    cb = 64 if case["fmt"] == "int8" else 32
    held = 2 * H * cb + 4 * H + 12  # codes, scales, time and position of a token
    N, C = float(sh["n"].sum()), float(sh["m"].sum())
    if case["kind"] == "score":
        pairs = float((sh["m"] * (sh["n"] + 1)).sum())
        seen = float(sh["n"][sh["m"] > 0].sum())
        return {"bytes": seen * held + C * (3 * d * 2 + 8) + C * d * 2 + (C * H * 4 if case["lse"] else 0),
                "flops": 4.0 * d * pairs}
    wide = 2 * d * (2 if case["src"] == "bf16" else 4) + 12
    return {"bytes": N * (wide + held) * (2 if case["kind"] == "append" else 1), "flops": N * 2 * d * 4}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _kv(g, rows, H, dtype):
    """Keys or values as a projection of normalised activations gives them: channels of unequal
    scale, tokens of unequal norm."""
    chan = torch.exp(0.5 * torch.randn(1, H * DH, generator=g, device="cuda"))
    tok = torch.exp(0.3 * torch.randn(rows, 1, generator=g, device="cuda"))
    return (torch.randn(rows, H * DH, generator=g, device="cuda") * chan * tok).to(dtype)


def _times(g, n, B):
    """Seconds of each user's interactions, non-decreasing, ending before the request: requests of
    about three interactions, gaps of half a minute and of an hour."""
    N = int(n.sum())
    u = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.from_numpy(n).cuda(), output_size=N)
    far = torch.rand(N, generator=g, device="cuda") < 0.1
    gap = torch.rand(N, generator=g, device="cuda").clamp_min(1e-6).log().neg() * torch.where(far, 3600.0, 30.0)
    gap = torch.where(torch.rand(N, generator=g, device="cuda") < 0.66, torch.zeros_like(gap), gap).long()
    total = torch.cumsum(gap, 0)
    end = torch.cumsum(torch.from_numpy(n).cuda(), 0)
    return T_REQ - 60 - (total[(end - 1).clamp_min(0)[u]] - total if N else total), u


def prepare(case, seed):
    sh = _shape(case)
    H, B, fmt = case["H"], case["B"], case["fmt"]
    d = H * DH
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + case["shape_seed"] % 1000003)
    row = _layout(H, fmt)[3]
    n, m = sh["n"], sh["m"]
    N, R = int(n.sum()), max(1, sh["rows"])
    dev = dict(device="cuda")
    ts_rows, user = _times(g, n, B)
    first = torch.from_numpy(np.concatenate([[0], np.cumsum(n)])).cuda()
    pos_rows = (torch.arange(N, **dev) - first[user] + 1).int()
    s = dict(case=case, H=H, B=B, fmt=fmt, N=N, R=R,
             begin=torch.from_numpy(sh["begin"]).cuda(), n=torch.from_numpy(n.astype(np.int32)).cuda(),
             cache=torch.zeros(R, row, dtype=torch.uint8, **dev),
             err=torch.zeros(1, dtype=torch.int32, **dev))
    if case["kind"] == "append":
        # the source rows are a jagged token array's: each user's new rows, then rows that are not
        # written (its candidates), keys and values inside wider rows
        dt = torch.bfloat16 if case["src"] == "bf16" else torch.float32
        m_tail = 3
        T = N + m_tail * B
        src = first[:-1] + m_tail * torch.arange(B, **dev)
        wide = torch.empty(T, 3 * d + 64, dtype=dt, **dev)
        wide[:, d:2 * d] = _kv(g, T, H, dt)
        wide[:, 2 * d:3 * d] = _kv(g, T, H, dt)
        at = src[user] + torch.arange(N, **dev) - first[user]
        pos = torch.zeros(T, dtype=torch.int32, **dev)
        ts = torch.full((T,), T_REQ, dtype=torch.int64, **dev)
        pos[at], ts[at] = pos_rows, ts_rows
        s.update(k=wide[:, d:2 * d], v=wide[:, 2 * d:3 * d], stride=3 * d + 64, T=T, pos=pos, ts=ts, dtype=dt,
                 src_offsets=torch.cat([src, src.new_tensor([T])]).int(), out_offsets=first.int())
        return s
    dst = s["begin"][user] + torch.arange(N, **dev) - first[user]
    if N:
        s["cache"][dst] = _rows(_kv(g, N, H, torch.bfloat16), _kv(g, N, H, torch.bfloat16), pos_rows, ts_rows, H, fmt)
    if case["kind"] == "read":
        s.update(out_offsets=first.int(), dtype=torch.bfloat16 if case["src"] == "bf16" else torch.float32)
        return s
    C = int(m.sum())
    qkv = torch.zeros(C, 3 * d + 64, dtype=torch.bfloat16, **dev)
    qkv[:, :d] = torch.randn(C, d, generator=g, **dev).to(torch.bfloat16)
    qkv[:, d:2 * d] = _kv(g, C, H, torch.bfloat16)
    qkv[:, 2 * d:3 * d] = _kv(g, C, H, torch.bfloat16)
    slopes = [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]
    s.update(C=C, M=max(1, int(m.max())), L=max(1, int(n.max())), max_cand=int(m.max()), max_len=int(n.max()),
             qkv=qkv, stride=3 * d + 64, cand_offsets=torch.from_numpy(np.concatenate([[0], np.cumsum(m)]).astype(np.int32)).cuda(),
             ts_cand=torch.full((C,), T_REQ, dtype=torch.int64, **dev),
             slope_pos=[float(np.float32(x)) for x in slopes], slope_time=[float(np.float32(x / 3600.0)) for x in slopes],
             scale=1.0 / math.sqrt(DH))
    return s


# ------------------------------------------------------------------------------------------
# plain form
# ------------------------------------------------------------------------------------------

def _codes(x, H, fmt):
    """Codes (whole fp32 numbers) [N, H, 64] and scales (bf16) [N, H] of rows x [N, H * 64]."""
    x = x.to(torch.bfloat16).float().view(-1, H, DH)
    a = x.abs().amax(-1)
    if fmt == "int8":
        f, e = torch.frexp(a)
        e = (e - 7 + (f > 127.0 / 128.0)).clamp(-126, 121)
        e = torch.where(a == 0, torch.full_like(e, -126), e)
        scale, most = torch.ldexp(torch.ones_like(a), e), 127.0
    else:
        f, e = torch.frexp(a / 7.0)
        scale = torch.ldexp(torch.floor(f * 32.0 + 0.5) / 32.0, e).clamp(2.0 ** -126, 36.0 * 2.0 ** 120)
        most = 7.0
    scale = scale.to(torch.bfloat16)
    c = torch.floor(x.abs() / scale.float()[..., None] + 0.5).clamp_max(most) * torch.sign(x)
    return c, scale


def _rows(k, v, pos, ts, H, fmt):
    """Cache rows (bytes) of keys and values [N, H * 64] with their positions and times."""
    cb, scales, tail, row = _layout(H, fmt)
    N = k.shape[0]
    out = torch.zeros(N, row, dtype=torch.uint8, device=k.device)
    (ck, sk), (cv, sv) = _codes(k, H, fmt), _codes(v, H, fmt)
    c = torch.stack([ck, cv], 1)
    if fmt == "int8":
        b = (c + 128.0).to(torch.uint8)
    else:
        b = (c + 8.0).to(torch.uint8)
        b = b[..., 0::2] | (b[..., 1::2] << 4)
    out[:, :scales] = b.reshape(N, scales)
    out[:, scales:scales + 4 * H] = torch.stack([sk, sv], -1).view(torch.uint8).reshape(N, 4 * H)
    out[:, tail:tail + 8] = ts.view(N, 1).view(torch.uint8)
    out[:, tail + 8:tail + 12] = pos.view(N, 1).view(torch.uint8)
    return out


def _values(rows, H, fmt):
    """(k, v [N, H, 64] fp32, pos int32, ts int64) of cache rows (bytes)."""
    cb, scales, tail, _ = _layout(H, fmt)
    N = rows.shape[0]
    b = rows[:, :scales].reshape(N, 2, H, cb)
    if fmt == "int8":
        c = b.float() - 128.0
    else:
        c = torch.stack([b & 15, b >> 4], -1).reshape(N, 2, H, DH).float() - 8.0
    sc = rows[:, scales:scales + 4 * H].contiguous().view(torch.bfloat16).view(N, H, 2).float()
    x = c * sc.permute(0, 2, 1)[..., None]
    return (x[:, 0], x[:, 1], rows[:, tail + 8:tail + 12].contiguous().view(torch.int32).view(N),
            rows[:, tail:tail + 8].contiguous().view(torch.int64).view(N))


def _row_of(s, counts, total):
    """(user, index within the user) of each of `total` rows, `counts` of them a user's."""
    user = torch.repeat_interleave(torch.arange(s["B"], device="cuda"), counts, output_size=total)
    first = torch.cumsum(counts, 0) - counts
    return user, torch.arange(total, device="cuda") - first[user]


def _plain_append(s):
    user, i = _row_of(s, s["n"].long(), s["N"])
    src = s["src_offsets"].long()[user] + i
    s["cache"][s["begin"][user] + i] = _rows(s["k"][src], s["v"][src], s["pos"][src], s["ts"][src], s["H"], s["fmt"])


def _plain_read(s):
    user, i = _row_of(s, s["n"].long(), s["N"])
    k, v, pos, ts = _values(s["cache"][s["begin"][user] + i], s["H"], s["fmt"])
    d = s["H"] * DH
    return dict(k=k.reshape(-1, d).to(s["dtype"]), v=v.reshape(-1, d).to(s["dtype"]), pos=pos, ts=ts)


def _plain_score(s):
    H, B, M, L, d = s["H"], s["B"], s["M"], s["L"], s["H"] * DH
    n, m = s["n"].long(), s["cand_offsets"].diff().long()
    j = torch.arange(L, device="cuda")
    seen = j < n[:, None]
    at = (s["begin"][:, None] + j).clamp_max(s["R"] - 1).reshape(-1)
    k, v, pos, ts = _values(s["cache"][at], H, s["fmt"])
    k = k.view(B, L, H, DH).permute(0, 2, 3, 1)
    v = v.view(B, L, H, DH).masked_fill(~seen[:, :, None, None], 0.0).transpose(1, 2)
    c = (s["cand_offsets"][:-1, None].long() + torch.arange(M, device="cuda")).clamp_max(max(0, s["C"] - 1))
    rows = s["qkv"][c.reshape(-1), :3 * d].float().view(B, M, 3, H, DH).permute(2, 0, 3, 1, 4)
    q, kc, vc = rows[0], rows[1], rows[2]
    x = torch.matmul(q, k).mul_(s["scale"])
    gap_p = (n[:, None] + 1 - pos.view(B, L)).abs().float()
    gap_t = (s["ts_cand"][c][:, :, None] - ts.view(B, 1, L)).abs().float()
    slope_p = torch.tensor(s["slope_pos"], device="cuda").view(H, 1, 1)
    slope_t = torch.tensor(s["slope_time"], device="cuda").view(H, 1, 1)
    x -= slope_p * gap_p[:, None, None, :]
    x -= slope_t * gap_t[:, None]
    x.masked_fill_(~seen[:, None, None, :], -math.inf)
    x_self = (q * kc).sum(-1, keepdim=True) * s["scale"]
    top = torch.maximum(x.amax(-1, keepdim=True), x_self)
    p, p_self = x.sub_(top).exp_(), torch.exp(x_self - top)
    total = p.sum(-1, keepdim=True) + p_self
    o = (torch.matmul(p, v) + p_self * vc) / total
    user, i = _row_of(s, m, s["C"])
    o = o.transpose(1, 2).reshape(B * M, d)[user * M + i].to(torch.bfloat16)
    if not s["case"]["lse"]:
        return dict(o=o)
    lse = (top + torch.log(total)).permute(1, 0, 2, 3).reshape(H, B * M)[:, user * M + i]
    return dict(o=o, lse=lse)


# ------------------------------------------------------------------------------------------
# the library's calls
# ------------------------------------------------------------------------------------------

def _own_read(G, s):
    d = s["H"] * DH
    k = torch.empty(s["N"], d, dtype=s["dtype"], device="cuda")
    v = torch.empty(s["N"], d, dtype=s["dtype"], device="cuda")
    pos = torch.empty(s["N"], dtype=torch.int32, device="cuda")
    ts = torch.empty(s["N"], dtype=torch.int64, device="cuda")
    G.qcache_read(s["out_offsets"], None, s["cache"], s["begin"], k, v, d, s["H"], DH, pos, ts, FMTS[s["fmt"]], s["err"])
    return dict(k=k, v=v, pos=pos, ts=ts)


def _own_append(G, s):
    G.qcache_append(s["src_offsets"], s["n"], s["k"], s["v"], s["stride"], s["H"], DH, s["pos"], s["ts"],
                    s["cache"], s["begin"], FMTS[s["fmt"]], s["err"], T=s["T"])


def _own_score(G, s):
    H, d, C = s["H"], s["H"] * DH, s["C"]
    if "ws" not in s:  # the workspace that a server keeps
        need = G.attn_qcached_workspace_size(s["B"], C, H, DH, s["max_cand"], s["max_len"])
        s["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    o = torch.empty(C, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(H, C, dtype=torch.float32, device="cuda") if s["case"]["lse"] else None
    qkv = s["qkv"]
    G.attn_fwd_qcached(s["cand_offsets"], s["max_cand"], qkv, qkv[:, d:], qkv[:, 2 * d:], s["stride"], s["cache"],
                       s["begin"], s["n"], s["max_len"], s["ts_cand"], H, DH, s["slope_pos"], s["slope_time"],
                       s["scale"], o, d, lse, s["ws"], FMTS[s["fmt"]], s["err"], C=C)
    return dict(o=o) if lse is None else dict(o=o, lse=lse)


def run(state):
    kind = state["case"]["kind"]
    if own:
        from generative_ranking_recommendation_b200 import genrank as G

        if kind == "score":
            return _own_score(G, state)
        if kind == "append":
            _own_append(G, state)
        return _own_read(G, state)
    if kind == "score":
        return _plain_score(state)
    if kind == "append":
        _plain_append(state)
    return _plain_read(state)


# ------------------------------------------------------------------------------------------
# float64
# ------------------------------------------------------------------------------------------

def _two_to(e):
    """2^e for whole e in [-300, 200], to the last bit (a device's power function may be one off,
    which would move values that lie halfway between two codes)."""
    return torch.from_numpy(np.ldexp(1.0, np.arange(-300, 201))).to(e.device)[e.long() + 300]


def _quantised64(x, H, fmt):
    """The values that the cache stands for, from the definition of its scales and codes."""
    x = x.to(torch.bfloat16).double().view(-1, H, DH)
    top = x.abs().max(-1, keepdim=True).values
    if fmt == "int8":
        need = top / 127
        e = torch.ceil(torch.log2(need.clamp_min(1e-60)))
        e = torch.where(need > _two_to(e), e + 1, torch.where(need <= _two_to(e - 1), e - 1, e)).clamp(-126, 121)
        step, most = _two_to(e), 127
    else:
        need = top / 7
        unit = _two_to(torch.floor(torch.log2(need.clamp_min(1e-60))) - 4)
        step = (torch.floor(need / unit + 0.5) * unit).clamp(2.0 ** -126, 36 * 2.0 ** 120)
        most = 7
    return torch.where(x < 0, -1.0, 1.0) * torch.floor(x.abs() / step + 0.5).clamp_max(most) * step


def _dequantised64(rows, H, fmt):
    """(k, v [N, H, 64], pos, ts) from a cache's bytes, by whole-number arithmetic."""
    cb, scales, tail, _ = _layout(H, fmt)
    b = rows.to(torch.int64)
    two = b[:, :scales].view(-1, 2, H, cb)
    code = two - 128 if fmt == "int8" else torch.stack([two % 16 - 8, two // 16 - 8], -1).flatten(-2)
    s16 = (b[:, scales:scales + 4 * H:2] + 256 * b[:, scales + 1:scales + 4 * H:2]).view(-1, H, 2)
    step = torch.where(s16 // 128 % 256 > 0, (128 + s16 % 128).double() * _two_to(s16 // 128 % 256 - 134),
                       torch.zeros((), dtype=torch.float64, device=rows.device))
    x = code.double() * step.transpose(1, 2)[..., None]
    weight = 256 ** torch.arange(7, device=rows.device)
    return x[:, 0], x[:, 1], (b[:, tail + 8:tail + 12] * weight[:4]).sum(-1), (b[:, tail:tail + 7] * weight).sum(-1)


def exact(case, seed):
    s = prepare(case, seed)
    sh = _shape(case)
    H, fmt, d = case["H"], case["fmt"], case["H"] * DH
    n, m, begin = sh["n"].tolist(), sh["m"].tolist(), sh["begin"].tolist()
    if case["kind"] == "append":
        src = s["src_offsets"].tolist()
        at = torch.cat([torch.arange(a, a + x) for a, x in zip(src, n)]).cuda()
        return dict(k=_quantised64(s["k"][at], H, fmt).view(-1, d), v=_quantised64(s["v"][at], H, fmt).view(-1, d),
                    pos=s["pos"][at], ts=s["ts"][at])
    if case["kind"] == "read":
        at = torch.cat([torch.arange(a, a + x) for a, x in zip(begin, n)]).cuda()
        k, v, pos, ts = _dequantised64(s["cache"][at], H, fmt)
        return dict(k=k.reshape(-1, d), v=v.reshape(-1, d), pos=pos.int(), ts=ts)
    o = torch.empty(s["C"], d, dtype=torch.float64, device="cuda")
    lse = torch.empty(H, s["C"], dtype=torch.float64, device="cuda")
    sp = torch.tensor(s["slope_pos"], dtype=torch.float64, device="cuda").view(H, 1, 1)
    st = torch.tensor(s["slope_time"], dtype=torch.float64, device="cuda").view(H, 1, 1)
    c0 = 0
    for nu, mu, bu in zip(n, m, begin):
        if mu == 0:
            continue
        k, v, pos, ts = _dequantised64(s["cache"][bu:bu + nu], H, fmt)
        q, kc, vc = (x.transpose(0, 1) for x in s["qkv"][c0:c0 + mu, :3 * d].double().view(mu, 3, H, DH).unbind(1))
        dp = (nu + 1 - pos).abs().double()
        dt = (s["ts_cand"][c0:c0 + mu, None] - ts).abs().double()
        x = torch.cat([torch.einsum("hmd,jhd->hmj", q, k) * s["scale"] - sp * dp - st * dt,
                       torch.einsum("hmd,hmd->hm", q, kc)[..., None] * s["scale"]], -1)
        z = torch.logsumexp(x, -1, keepdim=True)
        w = torch.exp(x - z)
        out = torch.einsum("hmj,jhd->hmd", w[..., :-1], v) + w[..., -1:] * vc
        o[c0:c0 + mu] = out.transpose(0, 1).reshape(mu, d)
        lse[:, c0:c0 + mu] = z[..., 0]
        c0 += mu
    return dict(o=o, lse=lse) if case["lse"] else dict(o=o)
