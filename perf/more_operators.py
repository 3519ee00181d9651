"""Measured cases of what stands before and behind the attention of a decoding step, and of attention
under masks: the norm and rotary position of queries and keys, the store that applies them on the way
into the pool (16-bit and 8-bit), read-slot attention whose rows see a range of keys with capped
scores and a bias by distance (fixed and ragged batches), and the scores of tokens from logits.

With own = False, run() computes the operators from elementary torch operations in float32 (the
angles of rotations in float64); with own = True it makes the calls of the package.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E_MIN, E_MAX = -50, 38          # exponents of a row in an 8-bit pool
EPS = 1e-6                      # of the norms


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one request, queries and keys out of a fused projection: latency
        dict(name="rotate token 1 gqa", op="rotate", B=1, rows=1, hq=32, hkv=8, d=128, dtype="bf16", rd=128,
             inter=False, norm=True, fused=True, scaling="none", far=30000),
        # the rows of 16 requests before a probe: half of each head rotated, interleaved, long-context frequencies
        dict(name="rotate probe 16x1562 gqa", op="rotate", B=16, rows=1562, hq=28, hkv=4, d=128, dtype="bf16", rd=64,
             inter=True, norm=False, fused=True, scaling="yarn", far=130000),
        # the store of one 32-token decode block of a 4-request batch, multi-head attention
        dict(name="store block 4x32 mha", op="store", B=4, rows=32, hq=32, hkv=32, d=128, dtype="bf16", rd=128,
             inter=False, norm=False, fused=True, scaling="none", far=8192, page=256),
        # the store of a recompute point: anchors and own rows of 16 requests, normed, odd row count
        dict(name="store point 16x1205 gqa", op="store", B=16, rows=1205, hq=28, hkv=4, d=128, dtype="bf16", rd=128,
             inter=False, norm=True, fused=True, scaling="linear", far=30000, page=256),
        # a shared affix of 8191 tokens registered in an 8-bit pool and read back for its first probe
        dict(name="store affix 8191 8-bit", op="store8", B=1, rows=8191, hq=32, hkv=8, d=128, dtype="bf16", rd=128,
             inter=False, norm=True, fused=True, scaling="none", far=8192, page=256),
        # single tokens of 8 requests that see the last 4096 keys, capped scores: serving
        dict(name="tokens 8x1x8000 window cap", op="mask", B=8, n_q=1, T=8000, L=0, hq=32, hkv=8, d=128, dtype="bf16",
             page=256, mask="window", width=4096, cap=50.0, bias=False, drop=False, lens=None),
        # the prompts of two requests, causal
        dict(name="prompt 2x4096x4096 causal", op="mask", B=2, n_q=4096, T=4096, L=0, hq=32, hkv=8, d=128,
             dtype="bf16", page=256, mask="causal", width=0, cap=0.0, bias=False, drop=False, lens=None),
        # a recompute point of 16 requests under block-causal masks, capped scores
        dict(name="point 16x986x2624 blocks cap", op="mask", B=16, n_q=986, T=2624, L=2048, hq=28, hkv=4, d=128,
             dtype="bf16", page=256, mask="blocks", width=32, cap=30.0, bias=False, drop=False, lens=None),
        # a mixed batch: packed documents next to single tokens and an idle request, biased by distance, head dim 64
        dict(name="ragged 9x700x3000 documents bias", op="mask", B=9, n_q=700, T=3000, L=0, hq=16, hkv=4, d=64,
             dtype="bf16", page=64, mask="documents", width=400, cap=0.0, bias=True, drop=True, lens=11),
        # one position in float32: the chosen token, its entropy and 20 alternatives (latency)
        dict(name="score 1x32000 f32", op="score", rows=1, vocab=32000, dtype="f32", k=20, given=True, temp=1.0,
             pad=0),
        # the masked positions of 4 decode blocks: confidence of the likeliest token, and entropy
        dict(name="score 128x126464", op="score", rows=128, vocab=126464, dtype="bf16", k=1, given=False, temp=1.0,
             pad=0),
        # the tokens of prompts scored with 5 alternatives each, rows of an odd length in a padded buffer
        dict(name="score 4100x100003", op="score", rows=4100, vocab=100003, dtype="bf16", k=5, given=True, temp=0.7,
             pad=61),
    ]


HEADS = ((32, 32), (28, 4), (32, 8), (16, 16), (8, 1), (2, 2), (12, 4))


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("rotate", "store", "store", "store8", "mask", "mask", "mask", "mask", "score", "score"))
    hq, hkv = rng.choice(HEADS)
    d = rng.choice((128, 128, 128, 64))
    dtype = "f32" if rng.random() < 0.15 else "bf16"
    if op == "score":
        while True:
            rows, vocab = _log(rng, 1, 4100), _log(rng, 50, 160000)
            if rows * vocab <= 4.1e8:
                break
        return dict(op=op, rows=rows, vocab=vocab, dtype=dtype, k=rng.choice((0, 1, 2, 5, 20, 32)),
                    given=rng.random() < 0.7, temp=rng.choice((1.0, 1.0, 0.3, 0.7, 1.5)), pad=rng.choice((0, 0, 7, 64)))
    page = rng.choice((0, 16, 64, 256))
    if op != "mask":
        while True:
            B, rows = _log(rng, 1, 16), _log(rng, 1, 8191)
            if B * rows * (hq + 2 * hkv) * d * (2 if dtype == "bf16" else 1) <= 2e8:
                break
        case = dict(op=op, B=B, rows=rows, hq=hq, hkv=hkv, d=d, dtype=dtype, rd=rng.choice((d, d, d // 2, d // 4 + 4)),
                    inter=rng.random() < 0.4, norm=rng.random() < 0.6, fused=rng.random() < 0.6,
                    scaling=rng.choice(("none", "none", "linear", "ntk", "yarn", "bands")), far=_log(rng, 100, 1000000))
        return case if op == "rotate" else dict(case, page=page)
    ragged = rng.random() < 0.35
    while True:
        B = _log(rng, 1, 32 if ragged else 16)
        T = _log(rng, 1, 16000 if ragged else 8704)
        n_q = min(T, rng.choice((1, 1, 32, _log(rng, 2, 4096))))
        work = B * hq * n_q * T * d
        if work <= (2e9 if dtype == "f32" else 1.4e11) and B * hkv * T * d <= 4e8 and B * hq * n_q * T <= 1.1e9:
            break
    mask = rng.choice(("none", "causal", "window", "blocks", "prefix", "documents"))
    return dict(op=op, B=B, n_q=n_q, T=T, L=0 if ragged else rng.randint(0, T), hq=hq, hkv=hkv, d=d, dtype=dtype,
                page=page, mask=mask, width=32 if mask == "blocks" else _log(rng, 1, T),
                cap=rng.choice((0.0, 0.0, 20.0, 50.0)), bias=rng.random() < 0.3, drop=rng.random() < 0.2,
                lens=rng.randrange(1 << 20) if ragged else None)


# ------------------------------------------------------------------------------ geometry
def _lens(case):
    """Query rows and keys of each request."""
    B, n, T = case["B"], case["n_q"], case["T"]
    if case["lens"] is None:
        return [n] * B, [T] * B
    r = random.Random(case["lens"])
    keys = [T] + [_log(r, 1, T) for _ in range(B - 1)]
    rows = [n] + [min(t, r.choice((1, 1, _log(r, 1, n)))) for t in keys[1:]]
    if B > 2:
        rows[2] = 0                       # an idle request keeps its cache entries
    return rows, keys


def _ranges(case):
    """Logical positions of the query rows and the keys [lo, hi) that each sees, flat over the requests."""
    rows, keys = _lens(case)
    r = np.random.RandomState(B_SEED + case["T"])
    pos, lo, hi = [], [], []
    for n, T in zip(rows, keys):
        p = np.arange(T - n, T)           # the request's last positions
        a, z = np.zeros(n, np.int64), np.full(n, T)
        if case["mask"] == "causal":
            z = p + 1
        elif case["mask"] == "window":
            a, z = np.maximum(0, p + 1 - case["width"]), p + 1
        elif case["mask"] == "blocks":
            z = np.minimum(T, (p // case["width"] + 1) * case["width"])
        elif case["mask"] == "prefix":
            z = np.maximum(p + 1, min(T, case["width"]))
        elif case["mask"] == "documents":
            cuts = np.unique(np.concatenate(([0, T], r.randint(0, T + 1, T // case["width"]))))
            doc = np.searchsorted(cuts, p, side="right") - 1
            a, z = cuts[doc], cuts[doc + 1]
            pad = p % 97 == 96            # rows of padding see nothing
            a, z = np.where(pad, 0, a), np.where(pad, 0, z)
        pos.append(p), lo.append(a), hi.append(z)
    return tuple(np.concatenate(x) for x in (pos, lo, hi))


B_SEED = 20011


def _pages(n, page, g, first):
    """n slots from shuffled pages of `page` slots starting at `first` (page 0: in order), and the
    slot behind the last page."""
    if page == 0:
        return first + torch.arange(n, device="cuda"), first + n
    np_ = -(-n // page)
    i = torch.arange(n, device="cuda")
    order = torch.randperm(np_, generator=g, device="cuda")
    return first + order[i // page] * page + i % page, first + np_ * page


# ------------------------------------------------------------------------------ inputs
def _rows(shape, g, dt):
    """Rows of K, V or Q: heads of different magnitude and a spread between tokens."""
    spread = torch.exp(0.4 * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))
    return (torch.randn(shape, generator=g, device="cuda") * spread).to(dt)


def _scaling(case):
    """Base, factor and trained length of the case's frequencies."""
    return {"none": (10000.0, 1.0, 0), "linear": (10000.0, 4.0, 8192), "ntk": (10000.0, 4.0, 8192),
            "yarn": (500000.0, 16.0, 8192), "bands": (500000.0, 8.0, 8192)}[case["scaling"]]


def _frequencies(case):
    """Angle per position of each pair, float64, and the amplitude of the rotation."""
    base, s, n = _scaling(case)
    rd, kind = case["rd"], case["scaling"]
    if kind == "ntk":
        base *= s ** (rd / (rd - 2))
    f = base ** (-torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd)
    if kind == "linear":
        f = f / s
    if kind == "yarn":                    # full turns over the trained length: above 32 as it is, below 1 divided
        i = torch.arange(rd // 2, dtype=torch.float64, device="cuda")
        low, high = (rd * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32, 1))
        low, high = max(math.floor(low), 0), min(math.ceil(high), rd - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1
    if kind == "bands":                   # the same by wavelength, between 1 and 4 turns
        keep = ((n * f / (2 * math.pi) - 1) / (4 - 1)).clamp(0, 1)
        f = f / s * (1 - keep) + f * keep
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    op, dt = case["op"], DT[case["dtype"]]
    st = dict(case=case, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if op == "score":
        R, V = case["rows"], case["vocab"]
        buf = torch.empty((R, V + case["pad"]), dtype=dt, device="cuda")
        for a in range(0, R, 512):
            x = 2.5 * torch.randn((min(512, R - a), V + case["pad"]), generator=g, device="cuda")
            top = torch.randint(0, V, (x.shape[0], 1), generator=g, device="cuda")
            buf[a:a + 512] = x.scatter_add_(1, top, 14 * torch.rand(top.shape, generator=g, device="cuda"))
        st["logits"] = buf[:, :V]
        st["logits"][:, 3] = -math.inf    # a token that is never chosen
        if case["given"]:
            st["tokens"] = torch.randint(0, V, (R,), generator=g, device="cuda", dtype=torch.int32)
            st["logprob"] = torch.empty(R, device="cuda")
        st["entropy"] = torch.empty(R, device="cuda")
        if case["k"]:
            st["top"] = torch.empty((R, min(case["k"], V)), dtype=torch.int32, device="cuda")
            st["top_logprob"] = torch.empty((R, min(case["k"], V)), device="cuda")
        return st
    B, hq, hkv, d = case["B"], case["hq"], case["hkv"], case["d"]
    if op == "mask":
        L = case["L"]
        rows, keys = _lens(case)
        st["scale"] = d ** -0.5
        shared, priv0 = _pages(L, case["page"], g, 0)
        priv, n = _pages(sum(t - L for t in keys), case["page"], g, priv0)
        parts, at = [], 0
        for t in keys:
            parts.append(torch.cat((shared, priv[at:at + t - L])))
            at += t - L
        rs = torch.cat(parts).to(torch.int32)
        if case["drop"]:
            rs = torch.where(torch.rand(rs.shape, generator=g, device="cuda") < 0.3, torch.full_like(rs, -1), rs)
        pos, lo, hi = _ranges(case)
        if case["mask"] != "none":
            st["row_range"] = torch.from_numpy(np.stack((lo, hi), 1)).to(torch.int32).cuda()
        if case["bias"]:
            st["q_pos"] = torch.from_numpy(pos).to(torch.int32).cuda()
            st["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq)
        st["num_slots"] = max(n, 1)
        st["k_cache"], st["v_cache"] = (_rows((max(n, 1), hkv, d), g, dt) for _ in range(2))
        st["q"] = (1.5 * torch.randn((sum(rows), hq, d), generator=g, device="cuda")).to(dt)
        if case["lens"] is None:
            rs, st["q"] = rs.view(B, -1), st["q"].view(B, -1, hq, d)
        else:
            st["q_start"] = torch.tensor([sum(rows[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
            st["kv_start"] = torch.tensor([sum(keys[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
            st["total_q"] = sum(rows)
        st["read_slot"], st["out"] = rs, torch.empty_like(st["q"])
        return st
    n = case["rows"]
    if case["fused"]:                     # slices of one projection's output
        st["q"], st["k"], st["v"] = _rows((B, n, hq + 2 * hkv, d), g, dt).split((hq, hkv, hkv), 2)
    else:
        st["q"], st["k"], st["v"] = (_rows((B, n, h, d), g, dt) for h in (hq, hkv, hkv))
    st["pos"] = torch.randint(0, case["far"], (B, n), generator=g, device="cuda").sort(1)[0].to(torch.int32)
    st["q_weight"], st["k_weight"] = ((1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) if case["norm"]
                                      else None for _ in range(2))
    st["freq"], st["amplitude"] = _frequencies(case)
    st["q_out"] = torch.empty((B, n, hq, d), dtype=dt, device="cuda")
    if op == "rotate":
        st["k_out"] = torch.empty((B, n, hkv, d), dtype=dt, device="cuda")
        return st
    slots, st["num_slots"] = _pages(B * n, case["page"], g, 0)
    st["slot"] = slots.view(B, n).to(torch.int32)
    shape = (st["num_slots"], hkv, d)
    if op == "store":
        st["k_cache"], st["v_cache"] = (_rows(shape, g, dt) for _ in range(2))
        return st
    st["k_cache"], st["v_cache"] = (torch.zeros(shape, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    st["kv_scale"] = torch.zeros((st["num_slots"], hkv, 2), dtype=torch.uint8, device="cuda")
    st["k_view"], st["v_view"] = (torch.empty((B, n, hkv, d), dtype=dt, device="cuda") for _ in range(2))
    return st


# ------------------------------------------------------------------------------ plain forms
def _plain_rotate(x, w, st, case):
    """The normed and rotated rows x [B, n, H, d] in float32."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    angle = st["pos"].double()[..., None] * st["freq"]
    c, s = ((f(angle) * st["amplitude"]).float()[:, :, None] for f in (torch.cos, torch.sin))
    rd = case["rd"]
    if case["inter"]:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        turned = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        turned = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((turned, x[..., rd:]), -1)


def _quantise_rows(x):
    """e4m3 codes and biased exponent of each row of the float32 tensor x [..., d]."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = (e - 9 + (m > 0.875)).clamp(E_MIN, E_MAX).to(torch.int32)       # 448 = 0.875 * 2^9
    e = torch.where(m == 0, torch.full_like(e, E_MIN), e)
    up = ((127 - e) << 23).view(torch.float32)                           # 2^-e
    return (x * up[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _plain_attend(q, k, v, see, bias, cap, scale):
    """q [B, n, Hq, d], k and v [B, T, Hkv, d], see [B, n, T]: softmax over the keys that a row sees; a row
    that sees none gives zeros."""
    B, n, hq, d = q.shape
    hkv, T = k.shape[2], k.shape[1]
    qg = q.float().view(B, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d)
    s = (qg @ k.float().permute(0, 2, 3, 1)).mul_(scale).view(B, hkv, hq // hkv, n, T)
    if cap:
        s = s.div_(cap).tanh_().mul_(cap)
    if bias is not None:                               # [Hq], [B, n, T]
        s = s - bias[0].view(1, hkv, -1, 1, 1) * bias[1][:, None, None]
    s = s.masked_fill_(~see[:, None, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    v = torch.where(see.any(1)[:, :, None, None], v.float(), torch.zeros((), device="cuda"))
    o = (s.view(B, hkv, -1, T) @ v.permute(0, 2, 1, 3)) / s.sum(-1).view(B, hkv, -1, 1).clamp_min(1e-30)
    return o.view(B, hkv, hq // hkv, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, hq, d)


def _plain_mask(st, case):
    B, n, T, dt = case["B"], case["n_q"], case["T"], DT[case["dtype"]]
    i, t = torch.arange(n, device="cuda"), torch.arange(T, device="cuda")
    ragged = case["lens"] is not None
    qs = st["q_start"].long() if ragged else n * torch.arange(B + 1, device="cuda")
    ks = st["kv_start"].long() if ragged else T * torch.arange(B + 1, device="cuda")
    at_q = (qs[:-1, None] + i).clamp_max(st["q"].numel() // (case["hq"] * case["d"]) - 1)       # [B, n]
    at_k = (ks[:-1, None] + t).clamp_max(st["read_slot"].numel() - 1)                            # [B, T]
    rs = st["read_slot"].reshape(-1)[at_k]
    there = (t < (ks[1:] - ks[:-1])[:, None]) & (rs >= 0)
    see = there[:, None].expand(B, n, T)
    if "row_range" in st:
        r = st["row_range"][at_q]
        see = see & (t >= r[..., :1]) & (t < r[..., 1:])
    bias = (st["slopes"], (st["q_pos"][at_q][..., None] - t).abs().float()) if case["bias"] else None
    slot = rs.clamp_min(0).long()
    q = st["q"].view(-1, case["hq"], case["d"])
    o = _plain_attend(q[at_q], st["k_cache"][slot], st["v_cache"][slot], see, bias, case["cap"], st["scale"]).to(dt)
    if not ragged:
        return o
    r = torch.arange(st["total_q"], device="cuda")
    b = torch.searchsorted(qs[1:].contiguous(), r, right=True)              # the request of each row
    return o[b, r - qs[b]]


def _plain_score(st, case):
    x = st["logits"].float()
    y = x / case["temp"]
    lse = torch.logsumexp(y, 1)
    out = {}
    if case["given"]:
        out["logprob"] = y.gather(1, st["tokens"].long()[:, None])[:, 0] - lse
    y = y.sub_(lse[:, None])
    p = y.exp()
    out["entropy"] = -torch.where(p > 0, p * y, torch.zeros((), device="cuda")).sum(1)
    if case["k"]:                                      # the largest logits, the lower token first where they are equal
        bits = (x + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, bits ^ 0x7fffffff, bits) << 32
        order -= torch.arange(case["vocab"], device="cuda")
        top = order.topk(min(case["k"], case["vocab"]), 1).indices
        out["top"], out["top_logprob"] = top.to(torch.int32), y.gather(1, top)
    return out


def _plain(st, case):
    op, dt = case["op"], DT[case["dtype"]]
    if op == "mask":
        return _plain_mask(st, case)
    if op == "score":
        return _plain_score(st, case)
    q = _plain_rotate(st["q"], st["q_weight"], st, case).to(dt)
    k = _plain_rotate(st["k"], st["k_weight"], st, case)
    if op == "rotate":
        return {"q": q, "k": k.to(dt)}
    slot = st["slot"].long()
    if op == "store":
        st["k_cache"][slot] = k.to(dt)
        st["v_cache"][slot] = st["v"]
        return {"q": q, "k": st["k_cache"], "v": st["v_cache"]}
    out = {"q": q}
    for i, (name, x) in enumerate((("k", k), ("v", st["v"].float()))):
        codes, exps = _quantise_rows(x)
        st[name + "_cache"].view(torch.uint8)[slot] = codes.view(torch.uint8)
        st["kv_scale"][slot, :, i] = exps
        factor = (st["kv_scale"][slot][..., i].to(torch.int32) << 23).view(torch.float32)
        out[name] = (st[name + "_cache"].view(torch.uint8)[slot].view(torch.float8_e4m3fn).float() * factor[..., None]).to(dt)
    return out


# ------------------------------------------------------------------------------ the package's calls
def _own(st, case):
    import affix_kv_cache_gb300 as ac
    op = case["op"]
    if op == "score":
        ac.acache_token_scores(case["rows"], case["vocab"], st["logits"], tokens=st.get("tokens"),
                               token_logprob=st.get("logprob"), entropy=st["entropy"], top_tokens=st.get("top"),
                               top_logprob=st.get("top_logprob"), temperature=case["temp"], dev_status=st["status"])
        return {n: st[n] for n in ("logprob", "entropy", "top", "top_logprob") if n in st}
    B, hkv = case["B"], case["hkv"]
    if "desc" not in st:                               # a program keeps both
        st["desc"] = ac.attn_desc(case["hq"], hkv, case["d"], case["d"] ** -0.5, case["dtype"])
        if op != "mask":
            base, factor, trained = _scaling(case)
            st["rope"] = ac.rope_desc(case["rd"], base, interleaved=case["inter"], scaling=case["scaling"],
                                      factor=factor, trained_len=trained)
    desc = st["desc"]
    if op == "mask":
        how = dict(row_range=st.get("row_range"), q_pos=st.get("q_pos"), slopes=st.get("slopes"), softcap=case["cap"],
                   drop_none=case["drop"], dev_status=st["status"])
        pool = (st["read_slot"], st["k_cache"], st["v_cache"], st["num_slots"], st["out"])
        if case["lens"] is None:
            ac.acache_slot_attention_masked(desc, B, case["n_q"], st["q"], case["T"], *pool, **how)
        else:
            ac.acache_slot_attention_masked_varlen(desc, B, st["q_start"], case["n_q"], st["total_q"], st["q"],
                                                   st["kv_start"], case["T"], *pool, **how)
        return st["out"]
    n = case["rows"]
    norm = dict(q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS)
    if op == "rotate":
        ac.acache_rotate_qk(desc, st["rope"], B * n, st["pos"], st["q"], st["k"], st["q_out"], st["k_out"], **norm)
        return {"q": st["q_out"], "k": st["k_out"]}
    new = (desc, st["rope"], B, n, st["pos"], st["slot"], st["q"], st["k"], st["v"], st["q_out"], st["k_cache"],
           st["v_cache"])
    if op == "store":
        ac.acache_rotate_store(*new, st["num_slots"], 0, **norm, dev_status=st["status"])
        return {"q": st["q_out"], "k": st["k_cache"], "v": st["v_cache"]}
    ac.acache_rotate_store_q8(*new, st["kv_scale"], st["num_slots"], 0, **norm, dev_status=st["status"])
    ac.acache_gather_slots_q8(desc, B, n, st["slot"], st["k_cache"], st["v_cache"], st["kv_scale"], st["num_slots"],
                              st["k_view"], st["v_view"], dev_status=st["status"])
    return {"q": st["q_out"], "k": st["k_view"], "v": st["v_view"]}


def run(st):
    if own:
        return _own(st, st["case"])
    return _plain(st, st["case"])


# ------------------------------------------------------------------------------ work
def work(case):
    """Every input byte read once (a slot that several rows or requests see once), every output byte
    written once; two multiply-adds per (row, key that it sees, element) of the attention."""
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "score":
        R, k = case["rows"], min(case["k"], case["vocab"])
        return {"bytes": R * (case["vocab"] * e + 8 * k + 4 + 8 * case["given"]), "flops": 0}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op != "mask":
        n = case["B"] * case["rows"]
        by = n * (4 + 2 * hq * d * e + hkv * d * e)                     # positions, queries, keys in
        if op == "rotate":
            return {"bytes": by + n * hkv * d * e, "flops": 0}
        by += n * (4 + hkv * d * e)                                     # slots, values in
        slot = 2 * hkv * (d * e if op == "store" else d + 1)
        return {"bytes": by + n * (slot if op == "store" else 2 * slot + 4 + 2 * hkv * d * e), "flops": 0}
    L, live = case["L"], 0.7 if case["drop"] else 1.0
    rows, keys = _lens(case)
    _, lo, hi = _ranges(case)
    shared, n_keys, n_map, at = np.zeros(L + 1, np.int64), 0, 0, 0
    for n, T in zip(rows, keys):
        edge = np.zeros(T + 1, np.int64)
        np.add.at(edge, lo[at:at + n], 1)
        np.add.at(edge, hi[at:at + n], -1)
        seen = np.cumsum(edge)[:T] > 0
        at += n
        shared[:min(L, T)] |= seen[:L]
        n_keys += int(seen[L:].sum())
        n_map += int(seen.sum())
    n_keys += int(shared.sum())
    by = n_keys * live * 2 * hkv * d * e + 4 * n_map + 2 * sum(rows) * hq * d * e
    by += 8 * sum(rows) * (case["mask"] != "none") + 4 * sum(rows) * case["bias"]
    return {"bytes": by, "flops": 4 * hq * d * int((hi - lo).sum()) * live}


# ------------------------------------------------------------------------------ 64 bits
def _exact_rows(x, w, pos, case):
    """Each pair of a normed row as a complex number, turned."""
    base, s, n = _scaling(case)
    rd, kind, pi = case["rd"], case["scaling"], math.pi
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    amplitude, freq = 1.0, []
    for i in range(rd // 2):
        if kind == "ntk":
            f = math.exp(-2 * i / rd * (math.log(base) + rd / (rd - 2) * math.log(s)))
        else:
            f = math.exp(-2 * i / rd * math.log(base))
        if kind == "linear":
            f /= s
        elif kind == "bands":
            turns = n * f / (2 * pi)                   # over the trained length
            f = f if turns > 4 else f / s if turns < 1 else f * ((turns - 1) / 3 + (4 - turns) / 3 / s)
        elif kind == "yarn":
            first, last = (rd / 2 * math.log(n / (2 * pi * t), base) for t in (32, 1))
            first, last = max(0, math.floor(first)), min(rd - 1, math.ceil(last))
            part = 0.0 if i <= first else 1.0 if i >= last else (i - first) / (last - first)
            f, amplitude = f * (1 - part + part / s), 1 + math.log(s) / 10
        freq.append(f)
    angle = pos.double()[..., None, None] * torch.tensor(freq, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.full_like(angle, amplitude), angle)
    y = x.clone()
    one, two = (slice(0, rd, 2), slice(1, rd, 2)) if case["inter"] else (slice(0, rd // 2), slice(rd // 2, rd))
    z = torch.complex(x[..., one], x[..., two]) * turn
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_codes(x):
    """Values of the rows x as e4m3 codes with a power of two: nearest, ties to even."""
    top = x.abs().amax(-1)
    e = torch.full_like(top, float(E_MIN))
    while bool((over := (top > 448 * torch.exp2(e)) & (e < E_MAX)).any()):
        e += over
    y = x / torch.exp2(e)[..., None]
    unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / unit) * unit * torch.exp2(e)[..., None]


def _exact_score(st, case):
    out = {n: [] for n in (("logprob",) if case["given"] else ()) + ("entropy",) + (("top", "top_logprob") if case["k"] else ())}
    for a in range(0, case["rows"], 64):
        x = st["logits"][a:a + 64].double()
        lp = torch.log_softmax(x / case["temp"], 1)
        out["entropy"].append(torch.special.entr(torch.softmax(x / case["temp"], 1)).sum(1))
        if case["given"]:
            out["logprob"].append(lp.gather(1, st["tokens"][a:a + 64, None].long())[:, 0])
        if case["k"]:
            at = x.sort(dim=1, descending=True, stable=True).indices[:, :case["k"]]
            out["top"].append(at.to(torch.int32))
            out["top_logprob"].append(lp.gather(1, at))
    return {n: torch.cat(v) for n, v in out.items()}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "score":
        return _exact_score(st, case)
    hq, hkv = case["hq"], case["hkv"]
    if op != "mask":
        q = _exact_rows(st["q"], st["q_weight"], st["pos"], case)
        k, v = _exact_rows(st["k"], st["k_weight"], st["pos"], case), st["v"].double()
        if op == "rotate":
            return {"q": q, "k": k}
        if op == "store8":
            return {"q": q, "k": _exact_codes(k), "v": _exact_codes(v)}
        pool = [st[n + "_cache"].double() for n in ("k", "v")]
        for p, x in zip(pool, (k, v)):
            p[st["slot"].long()] = x
        return {"q": q, "k": pool[0], "v": pool[1]}
    rows, keys = _lens(case)
    pos, lo, hi = (torch.from_numpy(x).cuda() for x in _ranges(case))
    q, rs = st["q"].reshape(-1, hq, case["d"]), st["read_slot"].reshape(-1)
    out, at, key0 = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), 0, 0
    for n, T in zip(rows, keys):
        sl = rs[key0:key0 + T].long()
        t = torch.nonzero(sl >= 0)[:, 0]               # positions whose key is there
        see = (t >= lo[at:at + n, None]) & (t < hi[at:at + n, None])
        away = (pos[at:at + n, None] - t).abs().double()
        for h in range(hq if n and len(t) else 0):
            kk, vv = (st[x][sl[t], h * hkv // hq].double() for x in ("k_cache", "v_cache"))
            s = q[at:at + n, h].double() @ kk.T * st["scale"]
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            if case["bias"]:
                s = s - 2.0 ** (-8 * (h + 1) / hq) * away
            s = torch.where(see, s, -math.inf)
            out[at:at + n, h] = torch.nan_to_num(torch.softmax(s, 1)) @ vv
        at, key0 = at + n, key0 + T
    return out.view(st["q"].shape)
