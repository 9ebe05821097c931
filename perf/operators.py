"""What is measured of the operators around a layer's attention over the paged cache.

Three operators, each with a plain form in elementary torch operations and, where `own` is
true, the call of the framework:

heads   the per-head norm of the new tokens' queries (and keys) and the position rotation,
        several tensors of the same tokens in one pass (``head_norm_rope``);
append  the new tokens' key, value and indexer-key rows, normed, rotated and stored in the
        paged pools in their formats, with the queries of the same tokens where a layer has
        them in hand at that point (``cache_append``);
attn    one decode step of exact attention over every cached position, for a batch that shares
        a long prefix: the prefix's pages are read once for the whole batch
        (``prefix_attn_decode``); a prefix of 0 is plain dense decode attention.

A case is drawn from its plain values alone; lengths follow from them, so that the work of a
case is known without its inputs, and only the values, the page order and the order of the rows
come from the seed.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
THETA = 10000.0
NOPE, KV, PE = 128, 512, 64      # latent heads: projected nope part, latent row, rotated part
I_ROPE = 64                      # rotated part of an indexer head of 128


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of the smallest decode workload (16 query heads of 128, one key head)
        {"name": "heads-token", "op": "heads", "kind": "gqa", "N": 1, "H": 16, "Hk": 1, "D": 128,
         "R": 128, "pos0": 4095},
        # one decode step of 32 sequences: rotated query parts into the latent queries, indexer
        # queries to FP8
        {"name": "heads-decode", "op": "heads", "kind": "latent", "N": 32, "H": 64, "Hi": 64,
         "Di": 128, "pos0": 8192},
        # a chunk of a prompt with grouped heads of an odd width, rotated in part, at far positions
        {"name": "heads-chunk", "op": "heads", "kind": "gqa", "N": 777, "H": 24, "Hk": 4, "D": 80,
         "R": 48, "pos0": 1000000},
        # a whole prompt of 16384 tokens, latent queries
        {"name": "heads-prompt", "op": "heads", "kind": "latent", "N": 16384, "H": 64, "Hi": 64,
         "Di": 128, "pos0": 0},
        # one decode step: 32 sequences each append one latent row and one FP8 indexer key; the
        # step's queries are prepared in the same call
        {"name": "append-step", "op": "append", "kind": "latent", "form": "append", "B": 32,
         "T": 1, "bs": 64, "Di": 128, "H": 64, "Hi": 64, "pos0": 8192},
        # separate K and V pools, four key heads, pages of 16, a few new tokens per sequence
        {"name": "append-tokens", "op": "append", "kind": "gqa", "form": "rows", "B": 9, "T": 5,
         "bs": 16, "Hk": 4, "D": 128, "R": 128, "Di": 64, "H": 0, "pos0": 4093},
        # a prompt of 16384 tokens stored at once
        {"name": "append-prompt", "op": "append", "kind": "latent", "form": "rows", "B": 1,
         "T": 16384, "bs": 64, "Di": 128, "H": 0, "Hi": 0, "pos0": 0},
        # a handful of short requests on 16 heads of 128 behind a common prompt of 2048
        {"name": "attn-tiny", "op": "attn", "B": 4, "H": 16, "Dk": 128, "Dv": 128, "latent": False,
         "bs": 64, "P": 2048, "lo": 1, "hi": 256},
        # dense decode without a common prefix, contexts up to the selection's K = 2048, where
        # every position would be selected
        {"name": "attn-dense", "op": "attn", "B": 32, "H": 64, "Dk": 576, "Dv": 512,
         "latent": True, "bs": 64, "P": 0, "lo": 1, "hi": 2048},
        # grouped-query sizes that are no powers of two, pages of 48, a prefix that ends in a page
        {"name": "attn-odd", "op": "attn", "B": 7, "H": 24, "Dk": 192, "Dv": 128, "latent": False,
         "bs": 48, "P": 5000, "lo": 0, "hi": 700},
        # the decode batch: 32 sequences behind a system prompt of 16384
        {"name": "attn-batch", "op": "attn", "B": 32, "H": 64, "Dk": 576, "Dv": 512,
         "latent": True, "bs": 64, "P": 16384, "lo": 1, "hi": 2048},
        # many requests on one long document
        {"name": "attn-document", "op": "attn", "B": 64, "H": 64, "Dk": 576, "Dv": 512,
         "latent": True, "bs": 64, "P": 65536, "lo": 16, "hi": 512},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["heads", "append", "attn"])
    if op == "heads":
        pos0 = rng.choice([0, 1, 4095, 131072, 1 << 20])
        if rng.random() < 0.5:
            return {"op": op, "kind": "latent", "N": _log(rng, 1, 8192), "H": rng.choice([8, 16, 64]),
                    "Hi": rng.choice([4, 32, 64]), "Di": 128, "pos0": pos0}
        D = 8 * rng.randint(4, 32)
        return {"op": op, "kind": "gqa", "N": _log(rng, 1, 8192), "H": rng.randint(1, 48),
                "Hk": rng.randint(1, 8), "D": D, "R": 2 * rng.randint(4, D // 2), "pos0": pos0}
    if op == "append":
        bs = rng.choice([1, 16, 48, 64, 128, 256])
        form = rng.choice(["append", "rows"])
        B = _log(rng, 1, 128)
        T = 1 if form == "append" else _log(rng, 1, max(1, 16384 // B))
        pos0 = rng.choice([0, 5, 1000, 65530])
        if rng.random() < 0.5:
            H = rng.choice([0, 16, 64]) if B * T <= 8192 else 0
            return {"op": op, "kind": "latent", "form": form, "B": B, "T": T, "bs": bs, "Di": 128,
                    "H": H, "Hi": H, "pos0": pos0}
        D = 8 * rng.randint(4, 32)
        return {"op": op, "kind": "gqa", "form": form, "B": B, "T": T, "bs": bs,
                "Hk": rng.randint(1, 8), "D": D, "R": 2 * rng.randint(4, D // 2),
                "Di": rng.choice([32, 64, 128]), "H": 0, "pos0": pos0}
    latent = rng.random() < 0.6
    B, P = _log(rng, 1, 64), rng.choice([0, _log(rng, 16, 32768)])
    Dk, Dv = (576, 512) if latent else (8 * rng.randint(4, 32), 8 * rng.randint(4, 32))
    return {"op": op, "B": B, "H": rng.choice([8, 16, 24, 40, 64]) if not latent else
            rng.choice([16, 32, 64]), "Dk": Dk, "Dv": Dv, "latent": latent,
            "bs": rng.choice([16, 32, 48, 64, 128]), "P": P, "lo": rng.choice([0, 1, 100]),
            "hi": _log(rng, 101, 2048 if P else 4096)}


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def _weight(g, n):
    return 1.0 + 0.1 * torch.randn(n, generator=g, device=DEV)


def _inv_freq(R):
    e = torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R
    return (THETA ** -e).to(torch.float32)


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], unevenly ordered, the ends among them."""
    if n == 1:
        return [hi]
    f = [(b * 0.6180339887498949) % 1.0 for b in range(n)]
    v = [lo + int(x * (hi - lo + 1)) for x in f]
    v[0], v[n // 2] = hi, lo
    return v


def _query_parts(c, g, N):
    """(x, spec, out) of the query tensors of N tokens."""
    if c["kind"] == "gqa":
        H, Hk, D, R = c["H"], c["Hk"], c["D"], c["R"]
        qkv = _randn(g, N, H + 2 * Hk, D)      # one fused projection; q and k are slices of it
        q, k = qkv[:, :H], qkv[:, H:H + Hk]
        spec = dict(norm="rms", norm_dim=D, eps=EPS, rope_offset=0, rope_dim=R, interleaved=False)
        freq = _inv_freq(R)
        return [(q, dict(spec, weight=_weight(g, D), inv_freq=freq), torch.empty_like(q, memory_format=torch.contiguous_format)),
                (k, dict(spec, weight=_weight(g, D), inv_freq=freq), torch.empty_like(k, memory_format=torch.contiguous_format))]
    H, Hi, Di = c["H"], c["Hi"], c["Di"]
    proj = _randn(g, N, H, NOPE + PE)
    qbuf = torch.zeros((N, H, KV + PE), dtype=torch.bfloat16, device=DEV)
    qi = _randn(g, N, Hi, Di)
    return [(proj[:, :, NOPE:], dict(norm="none", rope_offset=0, rope_dim=PE, interleaved=True,
                                     inv_freq=_inv_freq(PE)), qbuf[:, :, KV:]),
            (qi, dict(norm="rms", norm_dim=Di, eps=EPS, weight=_weight(g, Di), rope_offset=0,
                      rope_dim=I_ROPE, interleaved=False, inv_freq=_inv_freq(I_ROPE)),
             torch.empty((N, Hi, Di), dtype=torch.float8_e4m3fn, device=DEV))]


def _plans(parts):
    import sparse_attention_score_gb300 as dsa
    return dsa.HeadParts([dsa.HeadPart(x, out, **spec) for x, spec, out in parts])


def _prepare_heads(c, seed):
    g = _gen(seed)
    N = c["N"]
    parts = _query_parts(c, g, N)
    pos = (torch.arange(N, device=DEV) + c["pos0"]).to(torch.int32)
    s = {"op": "heads", "parts": parts, "pos": pos}
    if own:
        s["plan"] = _plans(parts)
    return s


def _prepare_append(c, seed):
    g = _gen(seed)
    B, T, bs, pos0 = c["B"], c["T"], c["bs"], c["pos0"]
    N = B * T
    ends = [pos0 + T + (b * 7) % 13 for b in range(B)]       # cached positions after the call
    starts = [e - T for e in ends]
    maxb = (max(ends) + bs - 1) // bs
    bt = np.full((B, maxb), -1, dtype=np.int32)
    slots = [(b, s) for b in range(B) for s in range(starts[b] // bs, (ends[b] - 1) // bs + 1)]
    nb = len(slots) + 2                                       # two pages stay unused
    perm = torch.randperm(nb, generator=g, device=DEV).cpu().numpy()
    for i, (b, s) in enumerate(slots):
        bt[b, s] = perm[i]
    seq = np.repeat(np.arange(B, dtype=np.int32), T)
    pos = np.concatenate([np.arange(s, s + T, dtype=np.int32) for s in starts])
    if c["form"] == "rows":
        order = torch.randperm(N, generator=g, device=DEV).cpu().numpy() if B > 1 else np.arange(N)
        seq, pos = seq[order], pos[order]
    dev = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    s = {"op": "append", "form": c["form"], "bs": bs, "nb": nb, "max_len": int(max(ends)),
         "bt": dev(bt), "lens": torch.tensor(ends, dtype=torch.int32, device=DEV),
         "seq": dev(seq), "pos": dev(pos)}
    Di = c["Di"]
    ki = _randn(g, N, 1, Di)
    ri = I_ROPE if Di == 128 else Di // 2
    ki_spec = dict(norm="layer", norm_dim=Di, eps=EPS, weight=_weight(g, Di),
                   bias=0.1 * torch.randn(Di, generator=g, device=DEV), rope_offset=0, rope_dim=ri,
                   interleaved=False, inv_freq=_inv_freq(ri))
    if c["kind"] == "latent":
        kv = _randn(g, N, 1, KV + PE)
        cache = [(kv, dict(norm="rms", norm_dim=KV, eps=EPS, weight=_weight(g, KV), rope_offset=KV,
                           rope_dim=PE, interleaved=True, inv_freq=_inv_freq(PE)),
                  _randn(g, nb, bs, KV + PE)),
                 (ki, ki_spec, _randn(g, nb, bs, Di).to(torch.float8_e4m3fn))]
    else:
        Hk, D, R = c["Hk"], c["D"], c["R"]
        kv = _randn(g, N, 2 * Hk, D)
        cache = [(kv[:, :Hk], dict(norm="rms", norm_dim=D, eps=EPS, weight=_weight(g, D),
                                   rope_offset=0, rope_dim=R, interleaved=False,
                                   inv_freq=_inv_freq(R)), _randn(g, nb, bs, Hk * D)),
                 (kv[:, Hk:], dict(norm="none"), _randn(g, nb, bs, Hk * D)),
                 (ki, ki_spec, _randn(g, nb, bs, Di))]
    s["cache"] = cache
    s["parts"] = _query_parts(c, g, N) if c["H"] else []
    if own:
        import sparse_attention_score_gb300 as dsa
        s["layout"] = dsa.PagedLayout(s["bt"], s["lens"], bs, nb, s["max_len"])
        s["plan"] = _plans(cache)
        s["qplan"] = _plans(s["parts"]) if s["parts"] else None
        s["ws"] = dsa.workspace(dsa.cache_append_workspace_size())
    return s


def _prepare_attn(c, seed):
    g = _gen(seed)
    B, H, Dk, Dv, bs, P = c["B"], c["H"], c["Dk"], c["Dv"], c["bs"], c["P"]
    suf = _spread(B, c["lo"], c["hi"])
    lens = [P + n for n in suf]
    shared = P // bs                                          # whole pages of the prefix
    maxb = max(1, (max(lens) + bs - 1) // bs)
    own_pages = [max(0, (n + bs - 1) // bs - shared) for n in lens]
    nb = shared + sum(own_pages) + 1
    perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32).cpu().numpy()
    bt = np.full((B, maxb), -1, dtype=np.int32)
    bt[:, :shared] = perm[:shared]
    at = shared
    for b in range(B):
        bt[b, shared:shared + own_pages[b]] = perm[at:at + own_pages[b]]
        at += own_pages[b]
    kp = _randn(g, nb, bs, Dk)
    vp = kp if c["latent"] else _randn(g, nb, bs, Dv)
    if P % bs:  # the page the prefix ends in is every sequence's own, with the same rows
        first = torch.from_numpy(bt[:, shared].astype(np.int64)).to(DEV)
        kp[first, :P % bs] = kp[first[:1], :P % bs]
        if not c["latent"]:
            vp[first, :P % bs] = vp[first[:1], :P % bs]
    s = {"op": "attn", "B": B, "H": H, "Dk": Dk, "Dv": Dv, "bs": bs, "P": P,
         "max_len": int(max(lens)), "bt": torch.from_numpy(bt).to(DEV),
         "lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "kp": kp, "vp": vp,
         "q": _randn(g, B, H, Dk), "scale": float(np.float32(1.0 / math.sqrt(Dk)))}
    if own:
        import sparse_attention_score_gb300 as dsa
        s["layout"] = dsa.PagedLayout(s["bt"], s["lens"], bs, nb, s["max_len"])
        s["out"] = torch.empty((B, H, Dv), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((B, H), dtype=torch.float32, device=DEV)
        s["ws"] = dsa.workspace(dsa.prefix_attn_decode_workspace_size(B, H, Dk, Dv, P))
    return s


def prepare(case, seed):
    return {"heads": _prepare_heads, "append": _prepare_append,
            "attn": _prepare_attn}[case["op"]](case, seed)


# ------------------------------------------------------------------------------- plain forms
def _transform(x, pos, out_dtype, norm="none", norm_dim=0, eps=0.0, weight=None, bias=None,
               rope_offset=0, rope_dim=0, interleaved=False, inv_freq=None):
    """The transformed heads [N, H, D] of tokens at pos [N], in 32 bits, rounded once."""
    y = x.float()
    if norm != "none":
        h = y[..., :norm_dim]
        if norm == "layer":
            h = h - h.mean(-1, keepdim=True)
        h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + eps)
        if weight is not None:
            h = h * weight
        if bias is not None:
            h = h + bias
        y = torch.cat([h, y[..., norm_dim:]], -1)
    if rope_dim:
        # far positions: the angle is formed in 64 bits, its sine and cosine then rounded
        ang = pos.double()[:, None, None] * inv_freq.double()
        co, si = torch.cos(ang).float(), torch.sin(ang).float()
        r = y[..., rope_offset:rope_offset + rope_dim]
        if interleaved:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2)
        else:
            a, b = r[..., :rope_dim // 2], r[..., rope_dim // 2:]
            r = torch.cat([a * co - b * si, b * co + a * si], -1)
        y = torch.cat([y[..., :rope_offset], r, y[..., rope_offset + rope_dim:]], -1)
    if out_dtype == torch.float8_e4m3fn:
        y = y.clamp(-448.0, 448.0)
    return y.to(out_dtype)


def _plain_append(s):
    if s["form"] == "append":
        seq, pos = torch.arange(s["lens"].shape[0], device=DEV), s["lens"].long() - 1
    else:
        seq, pos = s["seq"].long(), s["pos"].long()
    page = s["bt"][seq, torch.div(pos, s["bs"], rounding_mode="floor")].long()
    row = page * s["bs"] + pos % s["bs"]
    # at most three pools (a value row has neither norm nor rotation) and two query tensors
    pools = [_store(pool, row, _transform(x, pos, pool.dtype, **spec)) for x, spec, pool in s["cache"]]
    return pools + [_transform(x, pos, out.dtype, **spec) for x, spec, out in s["parts"]]


def _store(pool, row, y):
    flat = pool.view(-1, pool.shape[-1])
    if pool.dtype == torch.float8_e4m3fn:  # stored as bytes: the indexed write needs no arithmetic
        flat.view(torch.uint8)[row] = y.flatten(1).view(torch.uint8)
    else:
        flat[row] = y.flatten(1)
    return pool


def _rows_of(s, lo, hi):
    """Physical rows [B, hi - lo] of positions lo..hi-1 of every sequence (0 where a table has
    no page), and which of them are cached."""
    pos = torch.arange(lo, hi, device=DEV)
    page = s["bt"][:, torch.div(pos, s["bs"], rounding_mode="floor")].long()
    there = pos[None, :] < s["lens"].long()[:, None]
    return torch.where(there, page * s["bs"] + pos % s["bs"], 0), there


def _plain_attn(s):
    B, H, Dk, Dv, P = s["B"], s["H"], s["Dk"], s["Dv"], s["P"]
    kf, vf = s["kp"].view(-1, s["kp"].shape[-1]), s["vp"].view(-1, s["vp"].shape[-1])
    q = s["q"].float() * s["scale"]
    # the prefix once for all rows of the batch, then each sequence's own positions
    pre, _ = _rows_of(s, 0, P)
    pre = pre[0]
    zp = (q.reshape(B * H, Dk) @ kf[pre].float().t()).view(B, H, P)
    rows, there = _rows_of(s, P, max(s["max_len"], P))
    zs = torch.einsum("bhd,bld->bhl", q, kf[rows].float())
    zs = zs.masked_fill(~there[:, None, :], -math.inf)
    z = torch.cat([zp, zs], -1)
    m = z.amax(-1, keepdim=True) if z.shape[-1] else z.new_full((B, H, 1), -math.inf)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(z - m)
    l = p.sum(-1, keepdim=True)
    vs = torch.where(there[:, :, None], vf[rows][..., :Dv].float(), 0.0)
    o = (p[..., :P].reshape(B * H, P) @ vf[pre][:, :Dv].float()).view(B, H, Dv)
    o = o + torch.einsum("bhl,bld->bhd", p[..., P:], vs)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    return o.to(torch.bfloat16), (m + torch.log(l))[..., 0]


def run(state):
    s = state
    if own:
        import sparse_attention_score_gb300 as dsa
        if s["op"] == "heads":
            dsa.head_norm_rope(s["plan"], s["pos"])
            return [out for _, _, out in s["parts"]]
        if s["op"] == "append":
            seq, pos = (s["seq"], s["pos"]) if s["form"] == "rows" else (None, None)
            dsa.cache_append(s["layout"], seq, pos, s["plan"], s["ws"], heads=s["qplan"])
            return [pool for _, _, pool in s["cache"]] + [out for _, _, out in s["parts"]]
        dsa.prefix_attn_decode(s["layout"], s["q"], s["kp"], s["vp"], s["P"], s["scale"], s["out"],
                               s["lse"], s["ws"])
        return s["out"], s["lse"]
    if s["op"] == "heads":
        return [_transform(x, s["pos"], out.dtype, **spec) for x, spec, out in s["parts"]]
    if s["op"] == "append":
        return _plain_append(s)
    return _plain_attn(s)


# ------------------------------------------------------------------------------- floors
def _head_work(elems, in_b, out_b):
    return elems * (in_b + out_b)


def work(case):
    c = case
    if c["op"] == "attn":
        suf = _spread(c["B"], c["lo"], c["hi"])
        pos = c["P"] + sum(suf)
        row = c["Dk"] if c["latent"] else c["Dk"] + c["Dv"]
        seen = c["B"] * c["P"] + sum(suf)
        return {"bytes": 2 * pos * row + 2 * c["B"] * c["H"] * (c["Dk"] + c["Dv"]) + 4 * c["B"] * c["H"],
                "flops": 2 * seen * c["H"] * (c["Dk"] + c["Dv"])}
    N = c["N"] if c["op"] == "heads" else c["B"] * c["T"]
    elems4 = elems3 = 0                                       # bf16 to bf16, bf16 to e4m3
    if c["kind"] == "latent":
        elems4 += N * c["H"] * PE
        elems3 += N * c["Hi"] * c["Di"]
        if c["op"] == "append":
            elems4 += N * (KV + PE)
            elems3 += N * c["Di"]
    elif c["op"] == "heads":
        elems4 += N * (c["H"] + c["Hk"]) * c["D"]
    else:
        elems4 += N * (2 * c["Hk"] * c["D"] + c["Di"])
    n = elems4 + elems3
    return {"bytes": _head_work(elems4, 2, 2) + _head_work(elems3, 2, 1) + 8 * N, "flops": 10 * n}


# ------------------------------------------------------------------------------- 64 bits
def _exact_heads(x, pos, spec):
    y = x.double().clone()
    n = spec.get("norm_dim", 0)
    if spec["norm"] != "none":
        h = y[..., :n].clone()
        if spec["norm"] == "layer":
            h -= h.sum(-1, keepdim=True) / n
        h /= torch.sqrt(h.square().sum(-1, keepdim=True) / n + spec["eps"])
        y[..., :n] = h * spec["weight"].double()
        if spec.get("bias") is not None:
            y[..., :n] += spec["bias"].double()
    R, o = spec.get("rope_dim", 0), spec.get("rope_offset", 0)
    if R:
        i = torch.arange(R // 2, device=DEV)
        a, b = (o + 2 * i, o + 2 * i + 1) if spec["interleaved"] else (o + i, o + R // 2 + i)
        # a rotation is a product with a complex number of modulus 1
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           pos.double()[:, None] * spec["inv_freq"].double())[:, None, :]
        w = torch.complex(y[..., a], y[..., b]) * turn
        y[..., a], y[..., b] = w.real, w.imag
    return y


def _exact_pool(s, k):
    x, spec, pool = s["cache"][k]
    if s["form"] == "append":
        seq = list(range(s["lens"].shape[0]))
        pos = [int(n) - 1 for n in s["lens"].cpu()]
    else:
        seq, pos = s["seq"].cpu().tolist(), s["pos"].cpu().tolist()
    bt = s["bt"].cpu().numpy()
    want = pool.double()
    at = torch.tensor([[bt[b, p // s["bs"]], p % s["bs"]] for b, p in zip(seq, pos)], device=DEV).long()
    pos = torch.tensor(pos, device=DEV)
    want[at[:, 0], at[:, 1]] = _exact_heads(x, pos, spec).flatten(1)
    return want, pos


def _exact_attn(s):
    B, H, Dv, bs = s["B"], s["H"], s["Dv"], s["bs"]
    out = torch.zeros((B, H, Dv), dtype=torch.float64, device=DEV)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device=DEV)
    bt, lens = s["bt"].cpu(), s["lens"].cpu().tolist()
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        pages = bt[b, :(n + bs - 1) // bs].long().to(DEV)
        k = s["kp"][pages].flatten(0, 1)[:n].double()
        v = s["vp"][pages].flatten(0, 1)[:n, :Dv].double()
        z = (s["q"][b].double() @ k.t()) * s["scale"]
        lse[b] = torch.logsumexp(z, -1)
        out[b] = torch.softmax(z, -1) @ v
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "heads":
        return [_exact_heads(x, s["pos"], spec) for x, spec, _ in s["parts"]]
    if case["op"] == "append":
        pools = [_exact_pool(s, k) for k in range(len(s["cache"]))]
        return [p for p, _ in pools] + [_exact_heads(x, pools[0][1], spec) for x, spec, _ in s["parts"]]
    return _exact_attn(s)
