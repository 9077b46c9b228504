"""The operators around the attention, as they are timed and compared.

Five of them: the per-head norm with the position rotation (forward and
backward), the quantising write into a paged 8-bit cache, its read-back, and the
attention that reads the cache. `run` computes them in elementary torch
operations, or, where `own` is true, through the library's entry points.
"""

import math

import torch

own = False

ROPE_BASE = 10000.0
EPS = 1e-6
MIN_EXP, MAX_EXP = -100, 120  # exponents a cache scale may take

# The attention's key lengths and the cache's fill are spread over a batch by
# this fraction, so that a case fixes them without a seed.
GOLDEN = 0.6180339887498949


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one new token for each of 16 sequences, the smallest call of a decoding step
        dict(name="norm_rope_decode", op="norm_rope_fwd", B=16, Hq=32, Hkv=8, N=1, d=128, rot=128, interleaved=False,
             norm=True, far=131072),
        # a training batch, equal heads, from a packed projection
        dict(name="norm_rope_train", op="norm_rope_fwd", B=2, Hq=16, Hkv=16, N=8192, d=128, rot=128,
             interleaved=False, norm=True, far=8192),
        # the same batch's backward pass
        dict(name="norm_rope_bwd_train", op="norm_rope_bwd", B=2, Hq=16, Hkv=16, N=8192, d=128, rot=128,
             interleaved=False, norm=True, far=8192),
        # grouped heads, odd length, half of the head rotated, adjacent pairs
        dict(name="norm_rope_bwd_odd", op="norm_rope_bwd", B=3, Hq=8, Hkv=2, N=1237, d=64, rot=32, interleaved=True,
             norm=True, far=8192),
        # a decoding step's write: one token for each of 64 sequences, in the middle of their pages
        dict(name="append_decode", op="kv8_append", B=64, Hkv=8, d=128, page=64, n=1, L=4096, ragged=0.9, idle=0),
        # a prompt's write, ragged over the batch
        dict(name="append_prompt", op="kv8_append", B=4, Hkv=8, d=128, page=64, n=8192, L=8192, ragged=0.4, idle=0),
        # a long cache read back whole
        dict(name="gather_long", op="kv8_gather", B=4, Hkv=8, d=128, page=64, L=16384, ragged=0.0, idle=0),
        # a few short sequences in small pages, wide heads
        dict(name="gather_odd", op="kv8_gather", B=5, Hkv=2, d=256, page=16, L=777, ragged=0.7, idle=1),
        # a single short sequence: latency counts
        dict(name="decode_small", op="fwd_kv8", B=1, Hq=16, Hkv=4, Nq=1, d=128, page=16, L=1000, ragged=0.0, idle=0,
             causal=True),
        # decoding against long caches, grouped heads
        dict(name="decode_grouped", op="fwd_kv8", B=8, Hq=32, Hkv=8, Nq=1, d=128, page=64, L=32768, ragged=0.0, idle=0,
             causal=True),
        # a ragged decoding batch with equal heads, some slots without a sequence
        dict(name="decode_ragged", op="fwd_kv8", B=16, Hq=32, Hkv=32, Nq=1, d=64, page=32, L=8192, ragged=0.9, idle=2,
             causal=True),
        # a chunk of a prompt against what is cached so far
        dict(name="chunk_long", op="fwd_kv8", B=2, Hq=16, Hkv=4, Nq=1024, d=128, page=64, L=16384, ragged=0.3, idle=0,
             causal=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope_fwd", "norm_rope_bwd", "kv8_append", "kv8_gather", "fwd_kv8", "fwd_kv8"])
    d = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    g = rng.choice([1, 2, 3, 4, 8])
    if op.startswith("norm_rope"):
        most = (2 * 8192 * 48 * 128) // (Hkv * (g + 2) * d)  # tokens, for the training case's values
        N = min(_log(rng, 1, 16384), most)
        return dict(op=op, B=_log(rng, 1, min(64, most // N)), Hq=Hkv * g, Hkv=Hkv, N=N, d=d,
                    rot=rng.choice([16, d // 4 * 2, d, d]), interleaved=rng.random() < 0.3, norm=rng.random() < 0.8,
                    far=rng.choice([16384, 131072]))
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.choice([0.0, 0.3, 0.9])
    if op == "fwd_kv8":
        Nq = rng.choice([1, 1, 1, rng.randint(2, 16), _log(rng, 17, 1024)])
        L = _log(rng, Nq, 32768)
        most = (8 * 8 * 32768 * 128) // (L * Hkv * d)  # sequences, for the longest decoding case's cached values
        rows = (2 * 16 * 1024 * 16384 * 128) // (Hkv * g * L * d)  # queries, for the chunk's work
        Nq = min(Nq, rows)
        B = _log(rng, 1, min(32, most, rows // Nq))
        return dict(op=op, B=B, Hq=Hkv * g, Hkv=Hkv, Nq=Nq, d=d, page=page, L=L, ragged=ragged,
                    idle=1 if B > 2 and rng.random() < 0.3 else 0, causal=rng.random() < 0.8)
    L = _log(rng, 1, 16384)
    n = rng.choice([1, 1, _log(rng, 1, L)]) if op == "kv8_append" else 0
    B = _log(rng, 1, min(64, (4 * 8 * 16384 * 128) // (L * Hkv * d)))
    c = dict(op=op, B=B, Hkv=Hkv, d=d, page=page, L=L, ragged=ragged,
             idle=1 if B > 2 and rng.random() < 0.3 else 0)
    if op == "kv8_append":
        c["n"] = n
    return c


def _lens(c):
    """Keys of each sequence, the new ones among them; the last `idle` slots hold none."""
    out = []
    for b in range(c["B"]):
        f = (b * GOLDEN) % 1.0
        out.append(0 if b >= c["B"] - c["idle"] else max(1, int(round(c["L"] * (1.0 - c["ragged"] * f)))))
    return out


def _counts(c):
    """New tokens (queries) of each sequence: all of `n`, or as many as it holds."""
    n = c["n"] if c["op"] == "kv8_append" else c["Nq"]
    return [min(n, x) for x in _lens(c)]


def work(c):
    d = c["d"]
    if c["op"].startswith("norm_rope"):
        rows = c["B"] * c["N"]
        qk, v = rows * (c["Hq"] + c["Hkv"]) * d, rows * c["Hkv"] * d
        table = min(rows, c["far"]) * c["rot"] // 2 * 8 + rows * 4
        if c["op"] == "norm_rope_fwd":
            return {"bytes": 4 * (qk + v) + table, "flops": 8 * qk}
        return {"bytes": (6 if c["norm"] else 4) * qk + 4 * v + table, "flops": 16 * qk}
    lens = _lens(c)
    pages = sum(-(-x // c["page"]) for x in lens) * c["Hkv"]
    vals = sum(lens) * c["Hkv"] * d * 2
    small = pages * 8 + sum(-(-x // c["page"]) for x in lens) * 4 + c["B"] * 8
    if c["op"] == "kv8_append":
        new = sum(_counts(c)) * c["Hkv"] * d * 2
        touched = sum(-(-x // c["page"]) - (x - n) // c["page"] for x, n in zip(lens, _counts(c)) if n)
        return {"bytes": 3 * new + touched * (c["Hkv"] * 8 + 4) + c["B"] * 8, "flops": 3 * new}
    if c["op"] == "kv8_gather":
        return {"bytes": 3 * vals + small, "flops": vals}
    rows = sum(_counts(c)) * c["Hq"]
    pairs = 0
    for x, n in zip(lens, _counts(c)):
        pairs += c["Hq"] * (n * x - (n * (n - 1) // 2 if c["causal"] else 0))
    return {"bytes": vals + small + rows * (4 * d + 4), "flops": 4 * d * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _exp2i(e):
    """2**e for whole e in [-126, 127], exactly."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _scale_exp(amax):
    """The smallest e with amax <= 448 * 2**e, held within [MIN_EXP, MAX_EXP]."""
    m, x = torch.frexp(amax)
    return torch.where(amax > 0, x.to(torch.int32) - 9 + (m > 0.875).to(torch.int32), MIN_EXP).clamp(MIN_EXP, MAX_EXP)


def _cache(c, lens, g, dev):
    """A paged cache that holds lens[b] tokens: values of unit size with a spread over
    the heads, pages in a shuffled order, stale bytes where no token is."""
    B, Hkv, d, page = c["B"], c["Hkv"], c["d"], c["page"]
    max_pages = max(1, -(-c["L"] // page))
    need = [-(-x // page) for x in lens]
    total = B * max_pages + 3
    order = torch.randperm(total, generator=g, device=dev)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
    used = torch.arange(max_pages, device=dev)[None, :] < torch.tensor(need, device=dev)[:, None]
    table = torch.where(used, order[: B * max_pages].view(B, max_pages).to(torch.int32), table)
    out = []
    for _ in range(2):
        scale = torch.empty(total, Hkv, dtype=torch.float32, device=dev)
        code = torch.empty(total, Hkv, page, d, dtype=torch.uint8, device=dev)
        step = max(1, (1 << 27) // (Hkv * page * d))
        for p in range(0, total, step):
            q = min(total, p + step)
            spread = torch.exp2(2.0 * torch.randn(1, Hkv, 1, 1, generator=g, device=dev).clamp(-1, 1))
            x = torch.randn(q - p, Hkv, page, d, generator=g, device=dev) * spread.clamp(0.5, 2.0)
            s = _exp2i(_scale_exp(x.abs().amax((2, 3))))
            scale[p:q] = s
            code[p:q] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        out += [code, scale]
    # what lies behind a sequence's last token is whatever was there before
    last = [(b, need[b] - 1, lens[b] - (need[b] - 1) * page) for b in range(B) if lens[b] % page]
    if last:
        pid = table[[b for b, _, _ in last], [p for _, p, _ in last]].long()
        held = torch.tensor([n for _, _, n in last], device=dev)
        stale = (torch.arange(page, device=dev)[None, :] >= held[:, None])[:, None, :, None]
        junk = torch.randint(0, 256, (len(last), Hkv, page, d), generator=g, device=dev, dtype=torch.uint8)
        for code in (out[0], out[2]):
            code[pid] = torch.where(stale, junk, code[pid])
    return out, table


def prepare(c, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(int(seed) % (1 << 62))
    bf, f32 = torch.bfloat16, torch.float32

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(c=c, op=c["op"])
    d = c["d"]
    if c["op"].startswith("norm_rope"):
        B, Hq, Hkv, N, rot = c["B"], c["Hq"], c["Hkv"], c["N"], c["rot"]
        H = Hq + 2 * Hkv
        s["qkv"] = qkv = (randn(B, N, H, d) * 1.5).to(bf)  # a packed projection's output
        s["q_in"], s["k_in"], s["v_in"] = (t.transpose(1, 2) for t in qkv.split([Hq, Hkv, Hkv], dim=2))
        angle = torch.arange(c["far"], device=dev, dtype=torch.float64)[:, None] * torch.pow(
            torch.tensor(ROPE_BASE, device=dev, dtype=torch.float64),
            -torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)[None, :]
        s["cos"], s["sin"] = angle.cos().to(f32), angle.sin().to(f32)
        start = torch.randint(0, c["far"] - min(N, c["far"]) + 1, (B, 1), generator=g, device=dev)
        s["pos"] = ((start + torch.arange(N, device=dev)) % c["far"]).to(torch.int32)
        s["wq"] = 1 + 0.2 * randn(d) if c["norm"] else None
        s["wk"] = 1 + 0.2 * randn(d) if c["norm"] else None
        shapes = ((B, Hq, N, d), (B, Hkv, N, d), (B, Hkv, N, d))
        if c["op"] == "norm_rope_fwd":
            s["q"], s["k"], s["v"] = (torch.empty(x, dtype=bf, device=dev) for x in shapes)
        else:
            s["dq"], s["dk"], s["dv"] = (randn(*x).to(bf) for x in shapes)
            s["dqkv"] = torch.empty_like(qkv)
            s["dq_in"], s["dk_in"], s["dv_in"] = (t.transpose(1, 2) for t in s["dqkv"].split([Hq, Hkv, Hkv], dim=2))
            s["dwq"] = torch.empty(d, dtype=f32, device=dev) if c["norm"] else None
            s["dwk"] = torch.empty(d, dtype=f32, device=dev) if c["norm"] else None
            if own:
                import exact_softmax_attention_fa_gb300 as fa
                s["ws"] = torch.empty(max(1, fa.fa_norm_rope_bwd_workspace_size(B, Hq, Hkv, N, d)), dtype=torch.uint8,
                                      device=dev)
        return s

    lens, page, B, Hkv = _lens(c), c["page"], c["B"], c["Hkv"]
    (s["kc"], s["ks"], s["vc"], s["vs"]), s["table"] = _cache(c, lens, g, dev)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if c["op"] == "kv8_append":
        s["k"], s["v"] = (randn(B, Hkv, c["n"], d).to(bf) for _ in range(2))
        s["counts"] = torch.tensor(_counts(c), dtype=torch.int32, device=dev)
    elif c["op"] == "kv8_gather":
        s["k"], s["v"] = (torch.zeros(B, Hkv, c["L"], d, dtype=bf, device=dev) for _ in range(2))
    else:
        s["q"] = randn(B, c["Hq"], c["Nq"], d).to(bf)
        s["counts"] = torch.tensor(_counts(c), dtype=torch.int32, device=dev)
        s["o"] = torch.zeros(B, c["Hq"], c["Nq"], d, dtype=bf, device=dev)
        s["lse"] = torch.zeros(B, c["Hq"], c["Nq"], dtype=f32, device=dev)
        s["scale"] = 1.0 / math.sqrt(d)
        if own:
            import exact_softmax_attention_fa_gb300 as fa
            s["ws"] = torch.empty(max(1, fa.fa_fwd_kv8_workspace_size(B, c["Hq"], Hkv, c["Nq"], d)),
                                  dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    return _PLAIN[s["op"]](s)


def _own(s):
    import exact_softmax_attention_fa_gb300 as fa
    c = s["c"]
    if s["op"] == "norm_rope_fwd":
        fa.fa_norm_rope_fwd(s["q_in"], s["k_in"], s["v_in"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], s["q"],
                            s["k"], s["v"], interleaved=c["interleaved"], eps=EPS)
        return s["q"], s["k"], s["v"]
    if s["op"] == "norm_rope_bwd":
        fa.fa_norm_rope_bwd(s["dq"], s["dk"], s["dv"], s["q_in"], s["k_in"], s["wq"], s["wk"], s["cos"], s["sin"],
                            s["pos"], s["dq_in"], s["dk_in"], s["dv_in"], s["dwq"], s["dwk"], s["ws"],
                            interleaved=c["interleaved"], eps=EPS)
        return s["dqkv"], s["dwq"], s["dwk"]
    if s["op"] == "kv8_append":
        fa.fa_kv8_append(s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"],
                         counts=s["counts"])
        return s["kc"].view(torch.float8_e4m3fn), s["ks"], s["vc"].view(torch.float8_e4m3fn), s["vs"]
    if s["op"] == "kv8_gather":
        fa.fa_kv8_gather(s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["k"], s["v"])
        return s["k"], s["v"]
    fa.fa_fwd_kv8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["o"], s["lse"], c["causal"],
                  s["scale"], counts=s["counts"], workspace=s["ws"])
    return s["o"], s["lse"]


def _pairs(x, rot, interleaved):
    """The two members of each rotated pair, and what is not rotated."""
    r = x[..., :rot]
    if interleaved:
        return r[..., 0::2], r[..., 1::2], x[..., rot:]
    return r[..., : rot // 2], r[..., rot // 2:], x[..., rot:]


def _unpairs(a, b, rest, interleaved):
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _plain_norm_rope_fwd(s):
    c = s["c"]
    cos, sin = s["cos"][s["pos"].long()][:, None], s["sin"][s["pos"].long()][:, None]

    def one(x, w):
        z = x.float()
        if w is not None:
            z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS) * w
        a, b, rest = _pairs(z, c["rot"], c["interleaved"])
        return _unpairs(a * cos - b * sin, b * cos + a * sin, rest, c["interleaved"]).to(torch.bfloat16)

    return one(s["q_in"], s["wq"]), one(s["k_in"], s["wk"]), s["v_in"].contiguous()


def _plain_norm_rope_bwd(s):
    c = s["c"]
    cos, sin = s["cos"][s["pos"].long()][:, None], s["sin"][s["pos"].long()][:, None]

    def one(dy, x, w):
        a, b, rest = _pairs(dy.float(), c["rot"], c["interleaved"])
        g = _unpairs(a * cos + b * sin, b * cos - a * sin, rest, c["interleaved"])
        if w is None:
            return g.to(torch.bfloat16), None
        z = x.float()
        r = torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS)
        dw = (g * z * r).sum((0, 1, 2), dtype=torch.float64).float()
        h = g * w
        return (r * (h - z * r * r * (h * z).mean(-1, keepdim=True))).to(torch.bfloat16), dw

    dq, dwq = one(s["dq"], s["q_in"], s["wq"])
    dk, dwk = one(s["dk"], s["k_in"], s["wk"])
    return torch.cat([t.transpose(1, 2) for t in (dq, dk, s["dv"])], 2), dwq, dwk


def _plain_append(s):
    c = s["c"]
    B, Hkv, d, page, n = c["B"], c["Hkv"], c["d"], c["page"], c["n"]
    lens, counts = s["lens"].long(), s["counts"].long()
    start = lens - counts
    T = (n + page - 2) // page + 1  # pages that n tokens can touch
    dev = lens.device
    first = start // page
    at = first[:, None] * page + torch.arange(T * page, device=dev)  # the token each place of these pages holds
    new = (at >= start[:, None]) & (at < lens[:, None])
    old = at < start[:, None]
    touched = new.view(B, T, page).any(2)
    # a page that no new token reaches repeats the sequence's first one (or, for an idle sequence, one of the
    # first sequence with new tokens) and its contents
    t = torch.where(touched, torch.arange(T, device=dev)[None, :], 0)
    src_b = torch.where(counts > 0, torch.arange(B, device=dev), (counts > 0).long().argmax())
    pid = s["table"][src_b[:, None], (first[src_b][:, None] + t[src_b]).clamp(max=s["table"].shape[1] - 1)].long()
    sel = (src_b[:, None], t[src_b])

    def one(x, code, scale):
        row = (at - start[:, None]).clamp(0, n - 1)
        x = torch.take_along_dim(x.float(), row[:, None, :, None], 2).view(B, Hkv, T, page, d).transpose(1, 2)
        x, is_new, is_old = x[sel], new.view(B, T, page)[sel], old.view(B, T, page)[sel]  # [B, T, Hkv, page, d]
        finite = torch.isfinite(x) & is_new[:, :, None, :, None]
        s_new = _exp2i(_scale_exp(torch.where(finite, x.abs(), 0).amax((3, 4))))
        held = is_old.any(2)[:, :, None]
        s_old = scale[pid]
        sc = torch.where(held, torch.maximum(s_old, s_new), s_new)
        had = code[pid]
        had_f = had.view(torch.float8_e4m3fn).float()
        re = (had_f * (s_old / sc)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        x = torch.where(torch.isfinite(x), x / sc[..., None, None], float("nan"))
        enc = x.to(torch.float8_e4m3fn).view(torch.uint8)
        is_new, is_old = is_new[:, :, None, :, None], is_old[:, :, None, :, None]
        code[pid] = torch.where(is_new, enc, torch.where(is_old, re, had))
        scale[pid] = sc
        return code.view(torch.float8_e4m3fn), scale

    return (*one(s["k"], s["kc"], s["ks"]), *one(s["v"], s["vc"], s["vs"]))


def _rows(s, code, scale):
    """Every place of the sequences' pages as fp32 [B, Hkv, max_pages * page, d], zero where no token is."""
    c = s["c"]
    pid = s["table"].clamp(min=0).long()
    x = code[pid].view(torch.float8_e4m3fn).float() * scale[pid][..., None, None]
    B, P = pid.shape
    x = x.permute(0, 2, 1, 3, 4).reshape(B, c["Hkv"], P * c["page"], c["d"])
    held = torch.arange(P * c["page"], device=x.device)[None, :] < s["lens"][:, None]
    return torch.where(held[:, None, :, None], x, 0.0)


def _plain_gather(s):
    L = s["c"]["L"]
    return tuple(_rows(s, *t)[:, :, :L].to(torch.bfloat16) for t in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))


def _plain_fwd(s):
    c = s["c"]
    B, Hq, Hkv, Nq, d = c["B"], c["Hq"], c["Hkv"], c["Nq"], c["d"]
    k, v = _rows(s, s["kc"], s["ks"]), _rows(s, s["vc"], s["vs"])
    L, dev = k.shape[2], k.device
    lens, counts = s["lens"].long(), s["counts"].long()
    i, j = torch.arange(Nq, device=dev), torch.arange(L, device=dev)
    sees = j[None, None, :] < lens[:, None, None]
    if c["causal"]:
        sees = sees & (j[None, None, :] <= (lens - counts)[:, None, None] + i[None, :, None])
    sees = (sees & (i[None, :, None] < counts[:, None, None]))[:, None, None]  # [B, 1, 1, Nq, L]
    q = s["q"].float().view(B, Hkv, Hq // Hkv * Nq, d)
    t = (q @ k.transpose(2, 3) * s["scale"]).view(B, Hkv, Hq // Hkv, Nq, L)
    t = t.masked_fill(~sees, -math.inf)
    top = t.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(t - top)
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, -1, L) @ v).view(p.shape[:-1] + (d,)) / torch.where(l > 0, l, 1.0)
    lse = (torch.log(l) + top).squeeze(-1).view(B, Hq, Nq)
    o = o.view(B, Hq, Nq, d).to(torch.bfloat16)
    live = (i[None, :] < counts[:, None])[:, None]
    return torch.where(live[..., None], o, s["o"]), torch.where(live, lse, s["lse"])


_PLAIN = {"norm_rope_fwd": _plain_norm_rope_fwd, "norm_rope_bwd": _plain_norm_rope_bwd, "kv8_append": _plain_append,
          "kv8_gather": _plain_gather, "fwd_kv8": _plain_fwd}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(c, seed):
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    return {"norm_rope_fwd": _exact_norm_rope, "norm_rope_bwd": _exact_norm_rope, "kv8_append": _exact_append,
            "kv8_gather": _exact_gather, "fwd_kv8": _exact_fwd}[c["op"]](s)


def _exact_norm_rope(s):
    """The rotation as a product of complex numbers; the backward pass by its Jacobian."""
    c = s["c"]
    rot, f64 = c["rot"], torch.float64
    phase = torch.complex(s["cos"].to(f64), s["sin"].to(f64))[s["pos"].long()][:, None]  # [B, 1, N, rot / 2]

    def turn(x, ph):
        head, rest = x[..., :rot], x[..., rot:]
        if c["interleaved"]:
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * ph
            return torch.cat((torch.view_as_real(z).flatten(-2), rest), -1)
        z = torch.complex(head[..., : rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * ph
        return torch.cat((z.real, z.imag, rest), -1)

    def rms(x):
        return (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt()

    if c["op"] == "norm_rope_fwd":
        out = []
        for x, w in ((s["q_in"], s["wq"]), (s["k_in"], s["wk"])):
            x = x.to(f64)
            out.append(turn(x if w is None else x / rms(x) * w.to(f64), phase))
        return (*out, s["v_in"].to(f64).contiguous())
    dx, dws = [], []
    for dy, x, w in ((s["dq"], s["q_in"], s["wq"]), (s["dk"], s["k_in"], s["wk"])):
        gr = turn(dy.to(f64), phase.conj())
        if w is None:
            dx.append(gr)
            dws.append(None)
            continue
        u = x.to(f64)
        n = rms(u)
        hat = u / n
        dws.append(torch.einsum("bhnd,bhnd->d", gr, hat))
        gr = gr * w.to(f64)
        dx.append((gr - hat * torch.einsum("bhnd,bhnd->bhn", gr, hat)[..., None] / c["d"]) / n)
    dx.append(s["dv"].to(f64))
    return torch.cat([t.permute(0, 2, 1, 3) for t in dx], 2), dws[0], dws[1]


def _exact_append(s):
    """Values over their page's scale, before they are rounded to 8 bits; what else a page holds as it was."""
    c = s["c"]
    page = c["page"]
    out = []
    for x, code, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        val, sc = code.view(torch.float8_e4m3fn).float().double(), scale.double()
        for b, (end, n) in enumerate(zip(_lens(c), _counts(c))):
            start = end - n
            if n == 0:
                continue
            p0, p1 = start // page, (end - 1) // page
            pid = s["table"][b, p0: p1 + 1].long()
            P = p1 - p0 + 1
            lay = torch.zeros(c["Hkv"], P * page, c["d"], dtype=torch.float64, device=x.device)
            lay[:, start - p0 * page: end - p0 * page] = x[b, :, :n].double()
            lay = lay.view(c["Hkv"], P, page, c["d"]).transpose(0, 1)
            amax = lay.abs().amax((2, 3))
            e = torch.ceil(torch.log2(torch.where(amax > 0, amax, 1.0) / 448.0) - 1e-12)
            new = torch.where(amax > 0, torch.exp2(e.clamp(MIN_EXP, MAX_EXP)), 2.0 ** MIN_EXP)
            sc_p, held = new.clone(), start - p0 * page
            if held:
                sc_p[0] = torch.maximum(new[0], sc[pid[0]])
            was = val[pid]
            place = torch.arange(P * page, device=x.device).view(P, page) + p0 * page
            is_new = ((place >= start) & (place < end))[:, None, :, None]
            is_old = (place < start)[:, None, :, None]
            was = torch.where(is_old, was * (sc[pid] / sc_p)[..., None, None], was)
            val[pid] = torch.where(is_new, lay / sc_p[..., None, None], was)
            sc[pid] = sc_p
        out += [val, sc]
    return tuple(out)


def _exact_gather(s):
    c = s["c"]
    out = []
    for code, scale in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
        full = torch.zeros(c["B"], c["Hkv"], c["L"], c["d"], dtype=torch.float64, device=code.device)
        for b, n in enumerate(_lens(c)):
            if n:
                pid = s["table"][b, : -(-n // c["page"])].long()
                x = code[pid].view(torch.float8_e4m3fn).float().double() * scale[pid].double()[..., None, None]
                full[b, :, :n] = x.transpose(0, 1).reshape(c["Hkv"], -1, c["d"])[:, :n]
        out.append(full)
    return tuple(out)


def _exact_fwd(s):
    c = s["c"]
    Hkv, Nq, d = c["Hkv"], c["Nq"], c["d"]
    g = c["Hq"] // Hkv
    o, lse = s["o"].double(), s["lse"].double()
    for b, (L, n) in enumerate(zip(_lens(c), _counts(c))):
        if n == 0:
            continue
        pid = s["table"][b, : -(-L // c["page"])].long()
        place = torch.arange(L, device=o.device)
        # the first of a group's heads sit in one row block
        for h in range(Hkv):
            k, v = (t[pid, h].view(torch.float8_e4m3fn).float().double().mul_(sc[pid, h].double()[:, None, None])
                    .reshape(-1, d)[:L] for t, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            for u in range(h * g, (h + 1) * g):
                t = torch.einsum("nd,ld->nl", s["q"][b, u, :n].double(), k) * s["scale"]
                if c["causal"]:
                    late = place[None, :] > (L - n + torch.arange(n, device=o.device))[:, None]
                    t = t.masked_fill_(late, -math.inf)
                lse[b, u, :n] = torch.logsumexp(t, -1)
                o[b, u, :n] = torch.softmax(t, -1) @ v
    return o, lse
