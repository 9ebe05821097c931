"""Plain 64-bit forms of the new-token operators, and the bounds their tests use."""
import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}  # half a step, relative


def transform64(x, pos, norm="none", norm_dim=None, eps=1e-6, weight=None, bias=None,
                rope_offset=0, rope_dim=0, interleaved=False, inv_freq=None):
    """x [N, heads, dim] -> (exact values, a bound on what fp32 arithmetic may add).

    The norm's relative error is a few 2^-24 per step of its sums and the
    rotation's angle is good to 2^-21, so an element is off by at most
    2^-19 times the largest magnitude that enters it (its pair's, after the
    norm, or the bias's and the normed part's apart, which may cancel)."""
    y = x.double().cpu().clone()
    d = y.shape[-1]
    n = d if norm_dim is None else norm_dim
    amp = y.abs()
    if norm != "none":
        h = y[..., :n]
        if norm == "layer":
            # the mean is subtracted in fp32: its error is relative to the
            # elements before the subtraction
            scale = h.abs().amax(-1, keepdim=True)
            h = h - h.mean(-1, keepdim=True)
        else:
            scale = h.abs()
        r = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
        h, a = h * r, torch.maximum(scale, h.abs()) * r
        if weight is not None:
            h, a = h * weight.double().cpu(), a * weight.double().cpu().abs()
        if bias is not None:
            h, a = h + bias.double().cpu(), a + bias.double().cpu().abs()
        y[..., :n] = h
        amp = amp.clone()
        amp[..., :n] = a
    if rope_dim:
        t = pos.double().cpu()[:, None] * inv_freq.double().cpu()[None, :]
        co, si = torch.cos(t)[:, None, :], torch.sin(t)[:, None, :]
        k = torch.arange(rope_dim // 2)
        i, j = (2 * k, 2 * k + 1) if interleaved else (k, k + rope_dim // 2)
        i, j = i + rope_offset, j + rope_offset
        a, b = y[..., i].clone(), y[..., j].clone()
        y[..., i], y[..., j] = a * co - b * si, b * co + a * si
        s = amp[..., i] + amp[..., j]
        amp = amp.clone()
        amp[..., i], amp[..., j] = s, s
    return y, amp * 2.0 ** -19


def assert_heads_close(got, want, fp32, what=""):
    """One rounding to got's type on top of the fp32 error; E4M3 saturates, and
    its steps below 2^-6 are 2^-9."""
    if got.element_size() == 1:
        got = got.view(torch.float8_e4m3fn)
        want = want.clamp(-448.0, 448.0)
        tol = HALF[torch.float8_e4m3fn] * (want.abs() + fp32) + 2.0 ** -10 + fp32
    else:
        tol = HALF[torch.bfloat16] * (want.abs() + fp32) + fp32
    g = got.double().cpu()
    assert torch.equal(torch.isnan(g), torch.isnan(want)), f"{what}: NaNs differ"
    bad = ((g - want).abs() > tol) & ~torch.isnan(want)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} elements off, first at {bad.nonzero()[0].tolist()}: "
        f"{g[bad][0].item()} for {want[bad][0].item()} (tolerance {tol[bad][0].item()})")


def attend64(q, k_pool, v_pool, bt, lens, bs, num_blocks, prefix, sm_scale, Dv):
    """Exact attention of q [B, Hq, Dqk] over every cached position: (out, lse,
    sum of p |v|).  Positions behind a bad block id are left out.  The prefix
    is read through the table of the first sequence that has all of it."""
    B, Hq, Dqk = q.shape
    q, kp, vp = q.double().cpu(), k_pool.cpu(), v_pool.cpu()
    kp, vp = kp.reshape(-1, kp.shape[-1]), vp.reshape(-1, vp.shape[-1])
    bt, lens = np.asarray(bt), [min(int(n), bt.shape[1] * bs) for n in lens]
    src = next((b for b in range(B) if lens[b] >= prefix), -1)
    out = torch.zeros((B, Hq, Dv), dtype=torch.float64)
    mag = torch.zeros((B, Hq, Dv), dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    for b in range(B):
        p = np.arange(max(lens[b], 0))
        t = np.where((p < prefix) & (lens[b] >= prefix), src, b)
        page = bt[t, p // bs]
        ok = (page >= 0) & (page < num_blocks)
        rows = torch.from_numpy((page.astype(np.int64) * bs + p % bs)[ok])
        if not len(rows):
            continue
        k, v = kp[rows, :Dqk].double(), vp[rows, :Dv].double()
        z = (q[b] @ k.t()) * float(np.float32(sm_scale))
        w = torch.softmax(z, -1)
        out[b], mag[b], lse[b] = w @ v, w @ v.abs(), torch.logsumexp(z, -1)
    return out, lse, mag


def assert_attn_close(out, lse, want, lse_want, mag, what=""):
    """Weights rounded to bf16 once (each off by 2^-8 of itself, so the sum by
    2^-8 sum p |v|), scores and sums in fp32 (2^-12 covers 2 |dz| and 10,000
    additions), the result rounded to bf16 once.  lse: 1e-3, which 10,000
    fp32 additions (6e-4) and the scores' error stay inside."""
    g = out.double().cpu()
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -11) * mag
    bad = ~((g - want).abs() <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} elements off, first at "
        f"{bad.nonzero()[0].tolist()}: {g[bad][0].item()} for {want[bad][0].item()}")
    if lse is not None:
        l = lse.double().cpu()
        fin = torch.isfinite(lse_want)
        assert torch.equal(torch.isfinite(l), fin), f"{what}: lse finiteness"
        assert torch.equal(l[~fin], lse_want[~fin]), f"{what}: lse of empty rows"
        if bool(fin.any()):
            assert float((l[fin] - lse_want[fin]).abs().max()) <= 1e-3, f"{what}: lse"
