"""Cases for the operators around a paged KV cache: decode over pages, writing pages, prefill
with a sliding window and pinned first tokens, and the verification of drafted tokens.

A case is a dict with an "op": "decode" (one new token per sequence over bf16 or FP8 pages),
"append" (rotated K and V of new tokens into bf16 or FP8 pages), "prefill" (window plus first
tokens, whole sequences or a chunk after a cached prefix) and "verify" (accepted drafts and
the next token from given random numbers).
"""

import math

import torch

own = False

DQK, DV, ROT = 192, 128, 64          # head dims and rotated dims of the layers
E4M3_MAX = 448.0


def listed():
    return [
        # one short conversation on the sliding-window head layout: the latency of one call
        dict(name="decode_b1_short", op="decode", fp8=False, B=1, hq=64, hkv=8, lo=777, hi=777,
             page=16, window=0, first=0),
        # a full batch with ragged contexts on the global-attention layout
        dict(name="decode_b64_ragged", op="decode", fp8=False, B=64, hq=64, hkv=4, lo=1024, hi=16384,
             page=64, window=0, first=0),
        # a full batch bounded by a window, the first tokens pinned
        dict(name="decode_b64_window", op="decode", fp8=False, B=64, hq=64, hkv=8, lo=500, hi=16384,
             page=32, window=1024, first=4),
        # two long documents in FP8 pages: few rows, split over the length
        dict(name="decode_fp8_b2_long", op="decode", fp8=True, B=2, hq=64, hkv=4, lo=100001, hi=131072,
             page=128, window=0, first=0),
        # the cache write of one decode step
        dict(name="append_b64_step", op="append", fp8=False, B=64, hkv=8, n=1, lo=10, hi=200, page=16),
        # the cache write of a prompt chunk into FP8 pages
        dict(name="append_fp8_chunk", op="append", fp8=True, B=2, hkv=4, n=4096, lo=33, hi=1000, page=64),
        # a short prompt on one key/value head
        dict(name="prefill_short", op="prefill", B=1, n=203, off=0, rotated=False, hq=8, hkv=1,
             window=128, first=4),
        # the sliding-window layer over a long prompt, first tokens pinned
        dict(name="prefill_swa_32k", op="prefill", B=1, n=32768, off=0, rotated=False, hq=64, hkv=8,
             window=128, first=4),
        # the global layout bounded by a wide window, an attention prompt prefix pinned
        dict(name="prefill_wide_8k", op="prefill", B=1, n=8192, off=0, rotated=False, hq=64, hkv=4,
             window=2048, first=64),
        # one sequence, three drafts: the latency of one call
        dict(name="verify_b1", op="verify", B=1, T=3, V=32000, greedy=False, bf16=False),
        # a full batch, three drafts, a large vocabulary
        dict(name="verify_b64", op="verify", B=64, T=3, V=131072, greedy=False, bf16=False),
        # drafts taken by argmax (no draft distribution), bf16 probabilities, an odd vocabulary
        dict(name="verify_greedy_b16", op="verify", B=16, T=7, V=50021, greedy=True, bf16=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "append", "prefill", "prefill", "verify"])
    if kind == "decode":
        fp8 = rng.random() < 0.35
        hq, hkv = rng.choice([(64, 8), (64, 4), (8, 1), (32, 8), (16, 8), (8, 8)])
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, min(131072, 8_000_000 // (B * hkv * 2)))
        lo = max(1, int(hi * rng.uniform(0.05, 1.0)))
        window = 0 if rng.random() < 0.5 else _log(rng, 16, 4096)
        return dict(op="decode", fp8=fp8, B=B, hq=hq, hkv=hkv, lo=lo, hi=hi,
                    page=rng.choice([16, 24, 32, 64, 100, 128]), window=window,
                    first=rng.choice([0, 1, 4, 17, 64]) if window else 0)
    if kind == "append":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, 2000)
        return dict(op="append", fp8=rng.random() < 0.5, B=B, hkv=rng.choice([1, 4, 8]),
                    n=_log(rng, 1, max(1, 8192 // B)), lo=hi // 3, hi=hi, page=rng.choice([16, 24, 64, 128]))
    if kind == "prefill":
        hq, hkv, most = rng.choice([(64, 8, 16384), (64, 4, 8192), (8, 1, 16384), (32, 4, 16384), (16, 8, 8192)])
        B = rng.choice([1, 1, 2, 3])
        n = _log(rng, 1, most // B)
        off = rng.choice([0, 0, 16 * rng.randint(1, 128), rng.randint(1, 2048)])
        window = rng.choice([128, 128, _log(rng, 8, 129), _log(rng, 130, 2048)])
        return dict(op="prefill", B=B, n=n, off=off, rotated=off > 0 and rng.random() < 0.7, hq=hq, hkv=hkv,
                    window=window, first=rng.choice([1, 4, 4, 16, 33, 64, 128]))
    greedy = rng.random() < 0.3
    return dict(op="verify", B=_log(rng, 1, 64), T=rng.randint(0, 8), V=_log(rng, 500, 131072),
                greedy=greedy, bf16=rng.random() < 0.3)


def _lengths(c):
    """Ragged lengths over [lo, hi], the same for every seed (the work depends on them)."""
    return [c["lo"] + int((c["hi"] - c["lo"]) * ((0.5 + 0.6180339887498949 * b) % 1.0)) for b in range(c["B"])]


def _pages(c, lengths):
    return max(1, -(-max(lengths) // c["page"]))


def _theta(c):
    return 1.0e4 if c["hq"] // c["hkv"] <= 8 else 1.0e7


def _key_count(c, L):
    """Keys that the newest of L tokens sees."""
    lo = max(0, L - c["window"]) if c["window"] > 0 else 0
    return L - lo + min(c["first"], lo)


def work(case):
    c = case
    if c["op"] == "decode":
        keys = sum(_key_count(c, L) for L in _lengths(c))
        row = (DQK + DV) * (1 if c["fp8"] else 2) + (8 if c["fp8"] else 0)
        io = c["B"] * c["hq"] * ((DQK + DV) * 2 + 4)
        return {"bytes": keys * c["hkv"] * row + io, "flops": 2 * keys * c["hq"] * (DQK + DV)}
    if c["op"] == "append":
        rows = c["B"] * c["n"] * c["hkv"]
        return {"bytes": rows * ((DQK + DV) * (3 if c["fp8"] else 4) + (8 if c["fp8"] else 0)),
                "flops": rows * ROT * 3}
    if c["op"] == "prefill":
        n, off, W, F = c["n"], c["off"], c["window"], c["first"]
        pairs = sum(min(p + 1, W) + min(F, max(0, p - W + 1)) for p in range(off, off + n))
        keys = n + min(off, W - 1 + F)
        io = n * c["hq"] * (DQK + DV) * 2 + keys * c["hkv"] * (DQK + DV) * 2
        return {"bytes": c["B"] * io, "flops": 2 * c["B"] * c["hq"] * pairs * (DQK + DV)}
    rows = 1 if c["greedy"] else 2       # the target's row, and the draft's that is subtracted
    size = 2 if c["bf16"] else 4
    return {"bytes": c["B"] * (rows * c["V"] * size + (c["T"] + 1) * 8), "flops": c["B"] * c["V"] * 3}


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _fp8_rows(x):
    """E4M3 bytes and one scale per row (amax / 448) of x [..., D]."""
    scale = x.float().abs().amax(-1) / E4M3_MAX
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (x.float() / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("decode", "append"):
        lengths = _lengths(c)
        ahead = [L + c.get("n", 0) for L in lengths]
        width = _pages(c, ahead)
        n_pages = c["B"] * width + 3             # a pool with pages that no sequence holds
        s["table"] = torch.randperm(n_pages, generator=g, device="cuda")[: c["B"] * width].view(c["B"], width).int()
        s["k"] = _randn(g, n_pages, c["page"], c["hkv"], DQK)
        s["v"] = _randn(g, n_pages, c["page"], c["hkv"], DV)
        if c["fp8"]:
            s["k"], s["ks"] = _fp8_rows(s["k"])
            s["v"], s["vs"] = _fp8_rows(s["v"])
        s["len"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        if c["op"] == "decode":
            s["q"] = _randn(g, c["B"], c["hq"], DQK)
            s["sink"] = _randn(g, c["hq"], dtype=torch.float32)
        else:
            s["kn"] = _randn(g, c["B"], c["n"], c["hkv"], DQK)
            s["vn"] = _randn(g, c["B"], c["n"], c["hkv"], DV)
    elif c["op"] == "prefill":
        nk = c["off"] + c["n"]
        s["q"] = _randn(g, c["B"], c["n"], c["hq"], DQK)
        s["k"] = _randn(g, c["B"], nk, c["hkv"], DQK)
        s["v"] = _randn(g, c["B"], nk, c["hkv"], DV)
        s["sink"] = _randn(g, c["hq"], dtype=torch.float32)
    else:
        B, T, V = c["B"], c["T"], c["V"]
        dtype = torch.bfloat16 if c["bf16"] else torch.float32
        logits = torch.randn(B, T + 1, V, generator=g, device="cuda") * 3
        s["p"] = torch.softmax(logits, -1).to(dtype)
        near = logits[:, :T] + torch.randn(B, T, V, generator=g, device="cuda") * 0.7
        if c["greedy"]:
            s["draft"] = near.argmax(-1).int()
            s["qd"] = None
        else:
            s["qd"] = torch.softmax(near, -1).to(dtype)
            noise = -torch.log(-torch.log(torch.rand(B, T, V, generator=g, device="cuda").clamp(1e-12, 1 - 1e-7)))
            s["draft"] = (near + noise).argmax(-1).int()
        s["u"] = torch.rand(B, T + 1, generator=g, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _rope(x, pos, theta):
    """x [B, n, H, 192] fp32, pos [n] or [B, n]: rotate-half over the first ROT dims."""
    half = ROT // 2
    freq = theta ** (torch.arange(half, device=x.device, dtype=torch.float64) * (-2.0 / ROT))
    ang = pos.double()[..., None] * freq
    cos, sin = ang.cos().float()[..., None, :], ang.sin().float()[..., None, :]
    a, b = x[..., :half], x[..., half:ROT]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., ROT:]], -1)


def _rows_of(table, page, tok):
    """Pool rows of tokens tok [B, K] through the table [B, width]."""
    return table.long().gather(1, tok // page) * page + tok % page


def _sink_softmax(a, sink):
    """Weights of scores a [..., K] (masked places -inf) beside a sink score, and the log-sum."""
    m = torch.maximum(a.amax(-1, keepdim=True), sink)
    e = torch.exp(a - m)
    den = e.sum(-1, keepdim=True) + torch.exp(sink - m)
    return e / den, (m + torch.log(den)).squeeze(-1)


def _plain_decode(s):
    c = s["case"]
    B, hq, hkv = c["B"], c["hq"], c["hkv"]
    L = s["len"].long()[:, None]
    W, F = c["window"], c["first"]
    most = s["table"].shape[1] * c["page"]
    lo = (L - W).clamp(min=0) if W > 0 else torch.zeros_like(L)
    nf = lo.clamp(max=F)
    t = torch.arange(min(most, W + F) if W > 0 else most, device="cuda")[None]
    ok = t < nf + L - lo
    tok = torch.where(t < nf, t, lo + t - nf).clamp(max=most - 1)
    rows = _rows_of(s["table"], c["page"], tok)
    if c["fp8"]:
        k = s["k"].view(torch.float8_e4m3fn).view(-1, hkv, DQK)[rows].float() * s["ks"].view(-1, hkv)[rows][..., None]
        v = s["v"].view(torch.float8_e4m3fn).view(-1, hkv, DV)[rows].float() * s["vs"].view(-1, hkv)[rows][..., None]
    else:
        k = s["k"].view(-1, hkv, DQK)[rows].float()
        v = s["v"].view(-1, hkv, DV)[rows].float()
    q = s["q"].float().view(B, hkv, hq // hkv, DQK)
    a = torch.einsum("bhgd,bkhd->bhgk", q, k) * DQK ** -0.5
    a = a.masked_fill(~ok[:, None, None], -math.inf)
    w, lse = _sink_softmax(a, s["sink"].view(1, hkv, -1, 1))
    o = torch.einsum("bhgk,bkhd->bhgd", w, v)
    return o.reshape(B, hq, DV).bfloat16(), lse.reshape(B, hq)


def _plain_append(s):
    c = s["case"]
    pos = s["len"].long()[:, None] + torch.arange(c["n"], device="cuda")
    rows = _rows_of(s["table"], c["page"], pos)
    k = _rope(s["kn"].float(), pos, 1.0e4)
    v = s["vn"].float()
    if c["fp8"]:
        k8, ks = _fp8_rows(k)
        v8, vs = _fp8_rows(v)
        s["k"].view(-1, c["hkv"], DQK)[rows] = k8
        s["v"].view(-1, c["hkv"], DV)[rows] = v8
        s["ks"].view(-1, c["hkv"])[rows] = ks
        s["vs"].view(-1, c["hkv"])[rows] = vs
    else:
        s["k"].view(-1, c["hkv"], DQK)[rows] = k.bfloat16()
        s["v"].view(-1, c["hkv"], DV)[rows] = s["vn"]
    return _pools(s)


def _pools(s):
    if s["case"]["fp8"]:
        return s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn), s["ks"], s["vs"]
    return s["k"], s["v"]


def _plain_prefill(s):
    """Blocks of queries, each against the keys its windows span, and the first tokens."""
    c = s["case"]
    B, n, off, hkv, W, F = c["B"], c["n"], c["off"], c["hkv"], c["window"], c["first"]
    G, nk = c["hq"] // hkv, off + n
    pos_k = torch.arange(nk, device="cuda")
    q = _rope(s["q"].float(), off + torch.arange(n, device="cuda"), _theta(c))
    k = _rope(s["k"].float(), pos_k, _theta(c))
    if c["rotated"]:
        k = torch.where((pos_k < off)[:, None, None], s["k"].float(), k)
    v = s["v"].float()
    S = min(n, max(min(W, nk), 128))
    nb = -(-n // S)
    q = torch.nn.functional.pad(q, (0, 0, 0, 0, 0, nb * S - n)).view(B, nb, S, hkv, G, DQK)
    qpos = off + torch.arange(nb * S, device="cuda").view(nb, S, 1)
    span = min(S + W - 1, off + nb * S)
    kpos = (off + (torch.arange(nb, device="cuda") + 1) * S - span)[:, None] + torch.arange(span, device="cuda")
    lo = (qpos - W + 1).clamp(min=0)
    in_w = (kpos[:, None] >= lo) & (kpos[:, None] <= qpos) & (kpos[:, None] < nk)
    at = kpos.clamp(0, nk - 1)
    nf = min(F, nk)
    in_f = (torch.arange(nf, device="cuda") < lo).expand(nb, S, nf)
    a = torch.cat([torch.einsum("bnqhgd,bkhd->bnhgqk", q, k[:, :nf]),
                   torch.einsum("bnqhgd,bnkhd->bnhgqk", q, k[:, at])], -1) * DQK ** -0.5
    a.masked_fill_(~torch.cat([in_f, in_w], -1)[:, None, None], -math.inf)
    w, _ = _sink_softmax(a, s["sink"].view(hkv, G, 1, 1))
    o = torch.einsum("bnhgqk,bkhd->bnqhgd", w[..., :nf], v[:, :nf]) + \
        torch.einsum("bnhgqk,bnkhd->bnqhgd", w[..., nf:], v[:, at])
    return o.reshape(B, nb * S, c["hq"], DV)[:, :n].bfloat16().contiguous()


def _plain_verify(s):
    p, u, draft = s["p"], s["u"].double(), s["draft"].long()
    B, T = draft.shape
    at = torch.arange(B, device="cuda")
    px = p[:, :T].gather(2, draft[..., None])[..., 0].double()
    qx = torch.ones_like(px) if s["qd"] is None else s["qd"].gather(2, draft[..., None])[..., 0].double()
    count = (u[:, :T] * qx < px).long().cumprod(1).sum(1)
    row = p[at, count].double()
    less = count < T
    if T == 0:
        minus = torch.zeros_like(row)
    elif s["qd"] is None:
        minus = torch.zeros_like(row).scatter_(1, draft[at, count.clamp(max=T - 1)][:, None], less[:, None].double())
    else:
        minus = s["qd"][at, count.clamp(max=T - 1)].double() * less[:, None]
    rest = (row - minus).clamp(min=0)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, row)
    total = rest.cumsum(1)
    over = total > u[:, T:] * total[:, -1:]
    last = rest.shape[1] - 1 - (rest > 0).flip(1).int().argmax(1)
    token = torch.where(over.any(1), over.int().argmax(1), last)
    slot = torch.arange(T + 1, device="cuda")
    out = torch.where(slot < count[:, None], torch.nn.functional.pad(draft, (0, 1)), -1)
    out = torch.where(slot == count[:, None], token[:, None], out)
    return count.int(), out.int()


def run(state):
    s, c = state, state["case"]
    if own:
        from hybrid_sliding_window_sink_b200 import _lib
        if c["op"] == "decode":
            if c["fp8"]:
                return _lib.decode_paged_fp8(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["len"], s["sink"],
                                             window=c["window"], n_first=c["first"])
            return _lib.decode_paged(s["q"], s["k"], s["v"], s["table"], s["len"], s["sink"],
                                     window=c["window"], n_first=c["first"])
        if c["op"] == "append":
            if c["fp8"]:
                _lib.cache_append_paged_fp8(s["kn"], s["vn"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["len"],
                                            rope_theta=1.0e4, rot_dims=ROT)
            else:
                _lib.cache_append_paged(s["kn"], s["vn"], s["k"], s["v"], s["table"], s["len"],
                                        rope_theta=1.0e4, rot_dims=ROT)
            return _pools(s)
        if c["op"] == "prefill":
            return _lib.prefill_first(s["q"], s["k"], s["v"], s["sink"], window=c["window"], n_first=c["first"],
                                      pos_offset=c["off"], k_prefix_rotated=c["rotated"], rope_theta=_theta(c),
                                      rot_dims=ROT, want_lse=False)[0]
        return _lib.verify_drafts(s["p"], s["draft"], s["u"], s["qd"])
    return {"decode": _plain_decode, "append": _plain_append, "prefill": _plain_prefill,
            "verify": _plain_verify}[c["op"]](s)


# ------------------------------------------------------------------ 64 bits
def _turn64(x, pos, theta):
    """x [n, H, 192] double rotated at pos [n], as complex numbers x_d + i x_{d + ROT/2}."""
    half = ROT // 2
    z = torch.complex(x[..., :half], x[..., half:ROT])
    ang = pos.double()[:, None] / theta ** (torch.arange(half, device=x.device).double() / half)
    z = z * torch.polar(torch.ones_like(ang), ang)[:, None]
    return torch.cat([z.real, z.imag, x[..., ROT:]], -1)


def _value64(s, name, rows):
    x = s[name].flatten(0, 1)[rows]
    if s["case"]["fp8"]:
        return x.view(torch.float8_e4m3fn).double() * s[name + "s"].flatten(0, 1)[rows].double()[..., None]
    return x.double()


def _attend64(q, k, v, ok, sink):
    """q [m, d], k [K, d], v [K, dv], ok [m, K], sink: outputs and log-sums."""
    a = torch.where(ok, q @ k.T / math.sqrt(DQK), -math.inf)
    a = torch.cat([a, torch.full_like(a[:, :1], float(sink))], 1)
    lse = a.logsumexp(1)
    return torch.exp(a[:, :-1] - lse[:, None]) @ v, lse


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "decode":
        out, lse = torch.zeros(c["B"], c["hq"], DV).double(), torch.zeros(c["B"], c["hq"]).double()
        G = c["hq"] // c["hkv"]
        for b, L in enumerate(_lengths(c)):
            tok = [t for t in range(L) if c["window"] <= 0 or t >= L - c["window"] or t < c["first"]]
            tok = torch.tensor(tok, device="cuda")
            rows = s["table"][b][tok // c["page"]].long() * c["page"] + tok % c["page"]
            k, v = _value64(s, "k", rows), _value64(s, "v", rows)
            for h in range(c["hkv"]):
                for i in range(h * G, h * G + G):
                    o, l = _attend64(s["q"][b, i:i + 1].double(), k[:, h], v[:, h], tok[None] >= 0, s["sink"][i])
                    out[b, i], lse[b, i] = o[0].cpu(), l[0].cpu()
        return out, lse
    if c["op"] == "append":
        names = ("k", "v")
        pools = [s[x].view(torch.float8_e4m3fn).double() if c["fp8"] else s[x].double() for x in names]
        scales = [s["ks"].double(), s["vs"].double()] if c["fp8"] else []
        for b, L in enumerate(_lengths(c)):
            pos = L + torch.arange(c["n"], device="cuda")
            rows = s["table"][b][pos // c["page"]].long() * c["page"] + pos % c["page"]
            for i, x in enumerate((_turn64(s["kn"][b].double(), pos, 1.0e4), s["vn"][b].double())):
                if c["fp8"]:
                    top = x.abs().amax(-1) / E4M3_MAX
                    scales[i].view(-1, c["hkv"])[rows] = top
                    x = x / top[..., None]
                pools[i].view(-1, c["hkv"], x.shape[-1])[rows] = x
        return tuple(pools + scales)
    if c["op"] == "prefill":
        n, off, W, F = c["n"], c["off"], c["window"], c["first"]
        G, step = c["hq"] // c["hkv"], 1024
        out = torch.zeros(c["B"], n, c["hq"], DV, dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            pk = torch.arange(off + n, device="cuda")
            k = _turn64(s["k"][b].double(), pk, _theta(c))
            if c["rotated"]:
                k[:off] = s["k"][b, :off].double()
            q, v = _turn64(s["q"][b].double(), pk[off:], _theta(c)), s["v"][b].double()
            for i in range(0, n, step):
                j = min(n, i + step)
                keys = pk[max(0, off + i - W + 1):off + j]
                keys = torch.cat([pk[:min(F, int(keys[0]))], keys])
                pq = pk[off + i:off + j, None]
                ok = (keys <= pq) & ((keys > pq - W) | (keys < F))
                for h in range(c["hq"]):
                    out[b, i:j, h] = _attend64(q[i:j, h], k[keys, h // G], v[keys, h // G], ok, s["sink"][h])[0]
        return out
    counts, tokens = [], []
    p, u, draft = s["p"].double().cpu().numpy(), s["u"].double().cpu().numpy(), s["draft"].cpu().numpy()
    q = None if s["qd"] is None else s["qd"].double().cpu().numpy()
    for b in range(c["B"]):
        t = 0
        while t < c["T"] and u[b, t] * (1.0 if q is None else q[b, t, draft[b, t]]) < p[b, t, draft[b, t]]:
            t += 1
        rest = p[b, t].copy()
        if t < c["T"]:
            if q is None:
                rest[draft[b, t]] -= 1.0
            else:
                rest -= q[b, t]
        rest = rest.clip(min=0.0)
        rest = rest if rest.sum() > 0 else p[b, t]
        total = rest.cumsum()
        above = (total > u[b, c["T"]] * total[-1]).nonzero()[0]
        token = int(above[0]) if len(above) else int(rest.nonzero()[0][-1])
        counts.append(t)
        tokens.append(list(draft[b, :t]) + [token] + [-1] * (c["T"] - t))
    return torch.tensor(counts, dtype=torch.int32), torch.tensor(tokens, dtype=torch.int32)
