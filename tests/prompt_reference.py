"""Plain 64-bit forms of the packed prompt attention and of the 4-bit cache, and the bounds
their tests use."""
import math

import torch

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)          # magnitudes of E2M1 codes 0..7
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)             # between neighbours


def attend_prompt64(q, k, v, cu_q, cu_k, scale):
    """(out, lse, sum of p |v|) of every token of every sequence; a row takes part only with the
    keys that it sees, whatever the others hold."""
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    Nq, Hq, _ = q.shape
    G, Dv = Hq // k.shape[1], v.shape[2]
    scale = float(torch.tensor(scale, dtype=torch.float32))
    out = torch.zeros((Nq, Hq, Dv), dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((Nq, Hq), -math.inf, dtype=torch.float64)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        nq, nk = q1 - q0, k1 - k0
        if nq == 0 or nk == 0:
            continue
        see = (torch.arange(nq)[:, None] + nk - nq) >= torch.arange(nk)[None, :]
        some = see.any(-1)
        for h in range(Hq):
            kh, vh = k[k0:k1, h // G], v[k0:k1, h // G]
            z = (q[q0:q1, h] @ kh.t()) * scale
            odd = ~torch.isfinite(kh).all(-1)
            if bool(odd.any()):                            # 0 * NaN of a product is no key seen
                for j in odd.nonzero()[:, 0].tolist():
                    z[:, j] = (q[q0:q1, h] * kh[j]).sum(-1) * scale
            z = torch.where(see, z, -math.inf)
            l = torch.logsumexp(z, -1)
            w = torch.where(see, torch.exp(z - torch.where(some, l, 0.0)[:, None]), 0.0)
            fin = torch.where(torch.isfinite(vh), vh, 0.0)
            o = w @ fin
            for j, d in (~torch.isfinite(vh)).nonzero().tolist():
                o[:, d] = torch.where(see[:, j], o[:, d] + vh[j, d], o[:, d])
            out[q0:q1, h] = torch.where(some[:, None], o, 0.0)
            mag[q0:q1, h] = w @ fin.abs()
            lse[q0:q1, h] = torch.where(some, l, -math.inf)
    return out, lse, mag


def assert_rows_close(out, lse, want, lse_want, mag, weight, what="", floor=0.0):
    """A weight is off by at most `weight` of itself (half a step of its type), scores and sums in
    fp32 add at most 2^-11 of sum p |v| (2 |dz| with sums of 256 products and 10,000 additions),
    the result is rounded to bf16 once (2^-8).  floor: an absolute bound, for weights below their
    type's range.  lse: 1e-3, as for the other attentions."""
    g, w = out.double().cpu(), want
    fin = torch.isfinite(w)
    assert torch.equal(torch.isnan(g), torch.isnan(w)), f"{what}: NaNs differ"
    assert torch.equal(g[~fin & ~torch.isnan(w)], w[~fin & ~torch.isnan(w)]), f"{what}: infinities differ"
    tol = 2.0 ** -8 * w.abs() + (weight + 2.0 ** -11) * mag + floor
    bad = fin & ~((g - w).abs() <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
        f"{g[bad][0].item()} for {w[bad][0].item()} (tolerance {tol[bad][0].item()})")
    if lse is not None:
        l = lse.double().cpu()
        lfin = torch.isfinite(lse_want)
        assert torch.equal(l[~lfin & ~torch.isnan(lse_want)], lse_want[~lfin & ~torch.isnan(lse_want)]), what
        if bool(lfin.any()):
            assert float((l[lfin] - lse_want[lfin]).abs().max()) <= 1e-3, f"{what}: lse"


# ------------------------------------------------------------------------------- 4 bits
def quantise64(x, scale=None):
    """x [N, heads, D] bf16 -> (codes [N, heads, D], E4M3 scale bytes [N, heads, D / 16]).  Each
    comparison is exact: a midpoint times a group scale has 7 significant bits."""
    y = x.cpu().float()
    if scale is not None:
        y = y / scale.cpu().float()[:, None]               # one fp32 division
    y = y.unflatten(-1, (-1, 16))
    amax = y.abs().amax(-1, keepdim=True)
    s = torch.div(amax, torch.full_like(amax, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = torch.where(torch.isnan(amax), torch.tensor(0x7f, dtype=torch.uint8), s.view(torch.uint8))
    t, a = s.view(torch.float8_e4m3fn).double(), y.abs().double()
    c = torch.zeros(y.shape, dtype=torch.uint8)
    for i, m in enumerate(MIDS):                           # ties go to the even code
        c += (a > m * t) if i % 2 == 0 else (a >= m * t)
    c = torch.where(t > 0, c + 8 * torch.signbit(y).to(torch.uint8), torch.zeros_like(c))
    return c.flatten(-2), s[..., 0]


def pack_rows(kq, vq, nbytes):
    """Rows of the pool from (codes, scales) of K and V."""
    half = lambda c: c[..., 0::2] | (c[..., 1::2] << 4)  # noqa: E731
    row = torch.cat([half(kq[0]), half(vq[0]), kq[1], vq[1]], -1)
    return torch.nn.functional.pad(row, (0, nbytes - row.shape[-1]))


def values64(rows, Dk, Dv, ks=None, vs=None):
    """K and V in 64 bits of rows [..., heads, bytes]."""
    rows = rows.cpu()
    level = torch.tensor(LEVELS + tuple(-x for x in LEVELS), dtype=torch.float64)
    out = []
    for D, at, sc, hs in ((Dk, 0, (Dk + Dv) // 2, ks), (Dv, Dk // 2, (Dk + Dv) // 2 + Dk // 16, vs)):
        b = rows[..., at:at + D // 2]
        c = torch.stack([b & 15, b >> 4], -1).flatten(-2).long()
        t = rows[..., sc:sc + D // 16].contiguous().view(torch.float8_e4m3fn).double()
        x = (level[c].unflatten(-1, (-1, 16)) * t[..., None]).flatten(-2)
        out.append(x if hs is None else x * hs.cpu().double()[:, None])
    return out


def attend_cache64(q, pool, bt, lens, bs, nb, Dk, Dv, scale, ks=None, vs=None):
    """Exact attention of q [B, Hq, Dk] over the 4-bit pool: (out, lse, sum of p |v|, sum of |v|);
    positions behind a bad block id are left out."""
    q, pool = q.double().cpu(), pool.cpu()
    B, Hq, _ = q.shape
    Hk = pool.shape[1]
    scale = float(torch.tensor(scale, dtype=torch.float32))
    out = torch.zeros((B, Hq, Dv), dtype=torch.float64)
    mag, total = torch.zeros_like(out), torch.zeros_like(out)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    for b in range(B):
        p = torch.arange(max(int(lens[b]), 0))
        page = torch.as_tensor(bt)[b].long()[p // bs] if len(p) else p
        ok = (page >= 0) & (page < nb)
        if not bool(ok.any()):
            continue
        k, v = values64(pool[page[ok], :, (p % bs)[ok]], Dk, Dv, ks, vs)       # [n, Hk, D]
        for h in range(Hq):
            kh, vh = k[:, h // (Hq // Hk)], v[:, h // (Hq // Hk)]
            z = (kh @ q[b, h]) * scale
            lse[b, h] = torch.logsumexp(z, -1)
            w = torch.softmax(z, -1)
            out[b, h], mag[b, h], total[b, h] = w @ vh, w @ vh.abs(), vh.abs().sum(0)
    return out, lse, mag, total
