"""The operators of packed prompts, as they are timed and compared.

Four of them: the per-head norm with the rotation by several axes (forward and
backward), and the attention over packed sequences of different lengths (forward
and backward). `run` computes them in elementary torch operations, or, where
`own` is true, through the library's entry points.
"""

import math

import torch

own = False

ROPE_BASE = 10000.0
EPS = 1e-6

# The lengths of a batch are spread by this fraction, so that a case fixes them without a seed.
GOLDEN = 0.6180339887498949


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one new token for each of 16 sequences, the smallest call of a decoding step
        dict(name="axes_decode", op="axes_fwd", B=16, Hq=32, Hkv=8, N=1, d=128, sections="16,24,24", turns=False,
             interleaved=False, norm=True, far=131072),
        # a packed prompt of text, images and video
        dict(name="axes_prompt", op="axes_fwd", B=1, Hq=32, Hkv=8, N=16384, d=128, sections="16,24,24", turns=False,
             interleaved=False, norm=True, far=32768),
        # a training batch's backward pass, equal heads, the axes taking turns
        dict(name="axes_bwd_train", op="axes_bwd", B=2, Hq=16, Hkv=16, N=8192, d=128, sections="24,20,20", turns=True,
             interleaved=False, norm=True, far=8192),
        # image patches: height and width, adjacent pairs, part of a short head rotated, odd length
        dict(name="axes_bwd_odd", op="axes_bwd", B=3, Hq=8, Hkv=2, N=1237, d=64, sections="12,12", turns=False,
             interleaved=True, norm=True, far=8192),
        # three short prompts: latency counts
        dict(name="packed_small", op="packed_fwd", B=3, Hq=16, Hkv=4, d=128, L=200, ragged=0.9, empty=0, pad=0,
             causal=True),
        # a serving batch of many short prompts
        dict(name="packed_short", op="packed_fwd", B=256, Hq=32, Hkv=8, d=128, L=256, ragged=0.9, empty=0, pad=0,
             causal=True),
        # a batch of long prompts, one as long as all the short ones together
        dict(name="packed_prompt", op="packed_fwd", B=8, Hq=32, Hkv=8, d=128, L=8192, ragged=0.9, empty=0, pad=0,
             causal=True),
        # the patches of some images, every one sees every other; a slot without an image, padding behind the last
        dict(name="packed_patches", op="packed_fwd", B=24, Hq=16, Hkv=16, d=64, L=1369, ragged=0.6, empty=1, pad=77,
             causal=False),
        # the smallest training step: two documents just over a tile and under it
        dict(name="packed_bwd_small", op="packed_bwd", B=2, Hq=8, Hkv=8, d=128, L=129, ragged=0.9, empty=0, pad=0,
             causal=True),
        # a training batch of packed documents, grouped heads
        dict(name="packed_bwd_train", op="packed_bwd", B=8, Hq=16, Hkv=4, d=128, L=8192, ragged=0.9, empty=0, pad=0,
             causal=True),
        # many short documents, equal heads, padding behind the last
        dict(name="packed_bwd_short", op="packed_bwd", B=64, Hq=16, Hkv=16, d=64, L=512, ragged=0.9, empty=2, pad=33,
             causal=True),
        # wide heads, full attention, odd lengths
        dict(name="packed_bwd_wide", op="packed_bwd", B=3, Hq=8, Hkv=2, d=256, L=2501, ragged=0.5, empty=0, pad=0,
             causal=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["axes_fwd", "axes_bwd", "packed_fwd", "packed_fwd", "packed_bwd", "packed_bwd"])
    d = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    g = rng.choice([1, 2, 3, 4, 8])
    if op.startswith("axes"):
        most = (2 * 8192 * 48 * 128) // (Hkv * (g + 2) * d)  # tokens, for the training case's values
        N = min(_log(rng, 1, 16384), most)
        half = rng.choice([d // 4, d // 2, d // 2]) // 8 * 8
        axes = rng.choice([1, 2, 3, 3, 4])
        cuts = sorted(rng.sample(range(1, half), axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [half])]
        return dict(op=op, B=_log(rng, 1, min(64, most // N)), Hq=Hkv * g, Hkv=Hkv, N=N, d=d,
                    sections=",".join(map(str, sections)), turns=rng.random() < 0.4, interleaved=rng.random() < 0.3,
                    norm=rng.random() < 0.8, far=rng.choice([16384, 131072]))
    c = dict(op=op, B=_log(rng, 1, 512), Hq=Hkv * g, Hkv=Hkv, d=d, L=_log(rng, 1, 16384),
             ragged=rng.choice([0.0, 0.5, 0.9]), empty=0, pad=rng.choice([0, 0, rng.randint(1, 300)]),
             causal=rng.random() < 0.7)
    # as much as the long cases' products and rows
    most = 16 * 128 * 2e8 if op == "packed_bwd" else 32 * 128 * 2e8
    while True:
        lens = _lens(c)
        if c["Hq"] * d * sum(n * n for n in lens) <= most and (c["Hq"] + Hkv) * d * sum(lens) <= 2.2e8:
            break
        if c["B"] > 1:
            c["B"] = c["B"] * 2 // 3
        else:
            c["L"] = c["L"] * 2 // 3
    if c["B"] > 4 and rng.random() < 0.4:
        c["empty"] = rng.randint(1, 3)
    return c


def _lens(c):
    """The length of each sequence; the first `empty` ones of odd index hold no token."""
    out = []
    for b in range(c["B"]):
        f = (b * GOLDEN) % 1.0
        idle = b % 2 == 1 and b // 2 < c["empty"]
        out.append(0 if idle else max(1, int(round(c["L"] * (1.0 - c["ragged"] * f)))))
    return out


def _axes(c):
    """The axis that each rotated pair follows: in blocks, or taking turns until an axis has its share."""
    left = [int(x) for x in c["sections"].split(",")]
    if not c["turns"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out = []
    while any(left):
        for a, n in enumerate(left):
            if n:
                out.append(a)
                left[a] -= 1
    return out


def work(c):
    d = c["d"]
    if c["op"].startswith("axes"):
        rows, axes = c["B"] * c["N"], c["sections"].count(",") + 1
        rot = 2 * len(_axes(c))
        qk, v = rows * (c["Hq"] + c["Hkv"]) * d, rows * c["Hkv"] * d
        table = min(rows, c["far"]) * rot // 2 * 8 + rows * 4 * axes
        if c["op"] == "axes_fwd":
            return {"bytes": 4 * (qk + v) + table, "flops": 8 * qk}
        return {"bytes": (6 if c["norm"] else 4) * qk + 4 * v + table, "flops": 16 * qk}
    lens = _lens(c)
    T = sum(lens)
    pairs = sum(n * (n + 1) // 2 if c["causal"] else n * n for n in lens) * c["Hq"]
    heads = c["Hq"] + c["Hkv"]
    if c["op"] == "packed_fwd":
        return {"bytes": T * (4 * d * heads + 4 * c["Hq"]), "flops": 4 * d * pairs}
    return {"bytes": T * (8 * d * heads + 4 * c["Hq"]), "flops": 10 * d * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _positions(c, axes, g):
    """Positions [axes, B, N]: runs of text, where all axes count together, between images and
    clips, whose frames, rows and columns count from the position where they start."""
    B, N, far = c["B"], c["N"], c["far"]
    out = torch.zeros(axes, B, N, dtype=torch.int32)
    for b in range(B):
        p, at = int(torch.randint(0, max(1, far - N), (1,), generator=g)), 0
        while at < N:
            text, frames, rows, cols = torch.randint(1, 33, (4,), generator=g).tolist()
            text = torch.arange(4 * text).expand(axes, -1)
            frames = 1 + frames // 9
            grid = torch.stack([t.flatten() for t in torch.meshgrid(
                torch.arange(frames), torch.arange(rows), torch.arange(cols), indexing="ij")])
            grid = torch.cat((grid, grid[:1]))[(1 if axes == 2 else 0):][:axes] + 4 * text.shape[1] // 4
            both = torch.cat((text, grid), 1)[:, : N - at] + p
            out[:, b, at: at + both.shape[1]] = both % far
            at += both.shape[1]
            p = int(both.max()) + 1
    return out


def prepare(c, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(int(seed) % (1 << 62))
    bf, f32 = torch.bfloat16, torch.float32

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(c=c, op=c["op"])
    d, Hq, Hkv = c["d"], c["Hq"], c["Hkv"]
    H = Hq + 2 * Hkv
    if c["op"].startswith("axes"):
        B, N = c["B"], c["N"]
        s["qkv"] = qkv = (randn(B, N, H, d) * 1.5).to(bf)  # a packed projection's output
        s["q_in"], s["k_in"], s["v_in"] = (t.transpose(1, 2) for t in qkv.split([Hq, Hkv, Hkv], dim=2))
        s["axes"] = _axes(c)
        half = len(s["axes"])
        angle = torch.arange(c["far"], device=dev, dtype=torch.float64)[:, None] * torch.pow(
            torch.tensor(ROPE_BASE, device=dev, dtype=torch.float64),
            -torch.arange(half, device=dev, dtype=torch.float64) / half)[None, :]
        s["cos"], s["sin"] = angle.cos().to(f32), angle.sin().to(f32)
        host = torch.Generator().manual_seed(int(seed) % (1 << 62))
        s["pos"] = _positions(c, max(s["axes"]) + 1, host).to(dev)
        s["wq"] = 1 + 0.2 * randn(d) if c["norm"] else None
        s["wk"] = 1 + 0.2 * randn(d) if c["norm"] else None
        shapes = ((B, Hq, N, d), (B, Hkv, N, d), (B, Hkv, N, d))
        if c["op"] == "axes_fwd":
            s["q"], s["k"], s["v"] = (torch.empty(x, dtype=bf, device=dev) for x in shapes)
        else:
            s["dq"], s["dk"], s["dv"] = (randn(*x).to(bf) for x in shapes)
            s["dqkv"] = torch.empty_like(qkv)
            s["dq_in"], s["dk_in"], s["dv_in"] = (t.transpose(1, 2) for t in s["dqkv"].split([Hq, Hkv, Hkv], dim=2))
            s["dwq"] = torch.empty(d, dtype=f32, device=dev) if c["norm"] else None
            s["dwk"] = torch.empty(d, dtype=f32, device=dev) if c["norm"] else None
        if own:
            import exact_softmax_attention_fa_gb300 as fa
            s["axes"] = bytes(s["axes"])
            if c["op"] == "axes_bwd":
                s["ws"] = torch.empty(max(1, fa.fa_norm_rope_bwd_workspace_size(B, Hq, Hkv, N, d)), dtype=torch.uint8,
                                      device=dev)
        return s

    lens = _lens(c)
    T = sum(lens) + c["pad"]
    s["lens"] = lens
    s["cu"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
    s["scale"] = 1.0 / math.sqrt(d)
    s["qkv"] = (randn(T, H, d) * 1.5).to(bf)  # a packed projection's output: views of it are the inputs
    s["q"], s["k"], s["v"] = s["qkv"].split([Hq, Hkv, Hkv], dim=1)
    s["o"] = torch.zeros(T, Hq, d, dtype=bf, device=dev)
    s["lse"] = torch.zeros(Hq, T, dtype=f32, device=dev)
    if c["op"] == "packed_bwd":
        s["do"] = randn(T, Hq, d).to(bf)
        s["o"], s["lse"] = _plain_fwd(s)  # the forward's outputs, which the backward reads
        s["dqkv"] = torch.zeros_like(s["qkv"])
        s["dq"], s["dk"], s["dv"] = s["dqkv"].split([Hq, Hkv, Hkv], dim=1)
    if own:
        import exact_softmax_attention_fa_gb300 as fa
        s["plan"] = fa.PackedPlan(s["cu"], T, causal=c["causal"])  # once for all layers of a step
        if c["op"] == "packed_bwd":
            s["ws"] = torch.empty(max(1, fa.fa_bwd_packed_workspace_size(T, Hq, Hkv, d)), dtype=torch.uint8, device=dev)
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
    if s["op"] == "axes_fwd":
        fa.fa_norm_rope_axes_fwd(s["q_in"], s["k_in"], s["v_in"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"],
                                 s["axes"], s["q"], s["k"], s["v"], interleaved=c["interleaved"], eps=EPS)
        return s["q"], s["k"], s["v"]
    if s["op"] == "axes_bwd":
        fa.fa_norm_rope_axes_bwd(s["dq"], s["dk"], s["dv"], s["q_in"], s["k_in"], s["wq"], s["wk"], s["cos"], s["sin"],
                                 s["pos"], s["axes"], s["dq_in"], s["dk_in"], s["dv_in"], s["dwq"], s["dwk"], s["ws"],
                                 interleaved=c["interleaved"], eps=EPS)
        return s["dqkv"], s["dwq"], s["dwk"]
    if s["op"] == "packed_fwd":
        fa.fa_fwd_packed(s["q"], s["k"], s["v"], s["o"], s["lse"], s["plan"], c["causal"], s["scale"])
        return s["o"], s["lse"]
    fa.fa_bwd_packed(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["dq"], s["dk"], s["dv"], s["plan"],
                     c["causal"], s["scale"], s["ws"])
    return s["dqkv"]


def _pairs(x, rot, interleaved):
    """The two members of each rotated pair, and what is not rotated."""
    r = x[..., :rot]
    if interleaved:
        return r[..., 0::2], r[..., 1::2], x[..., rot:]
    return r[..., : rot // 2], r[..., rot // 2:], x[..., rot:]


def _unpairs(a, b, rest, interleaved):
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _angles(s):
    """Cosines and sines [B, 1, N, rot / 2] of every token's pairs, each at its own axis's position."""
    axis = torch.tensor(list(s["axes"]), device=s["pos"].device)
    at = s["pos"].long()[axis].permute(1, 2, 0)  # [B, N, rot / 2]
    return torch.take_along_dim(s["cos"][None], at, 1)[:, None], torch.take_along_dim(s["sin"][None], at, 1)[:, None]


def _plain_axes_fwd(s):
    c = s["c"]
    cos, sin = _angles(s)
    rot = 2 * cos.shape[-1]

    def one(x, w):
        z = x.float()
        if w is not None:
            z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS) * w
        a, b, rest = _pairs(z, rot, c["interleaved"])
        return _unpairs(a * cos - b * sin, b * cos + a * sin, rest, c["interleaved"]).to(torch.bfloat16)

    return one(s["q_in"], s["wq"]), one(s["k_in"], s["wk"]), s["v_in"].contiguous()


def _plain_axes_bwd(s):
    c = s["c"]
    cos, sin = _angles(s)
    rot = 2 * cos.shape[-1]

    def one(dy, x, w):
        a, b, rest = _pairs(dy.float(), rot, c["interleaved"])
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


def _parts(s):
    """(rows, K/V heads) of the pieces that the plain forms take at a time: a sequence, and as many
    of its heads as keep the scores within a few GB."""
    c, at = s["c"], 0
    for n in s["lens"]:
        if n:
            step = max(1, (1 << 29) // (c["Hq"] // c["Hkv"] * n * n))
            for h in range(0, c["Hkv"], step):
                yield slice(at, at + n), slice(h, min(c["Hkv"], h + step))
        at += n


def _scores(s, rows, kv):
    """Scores of a piece [K/V heads, g, n, n], masked, and its q, k, v by K/V head, in 32 bits."""
    c = s["c"]
    g, n = c["Hq"] // c["Hkv"], rows.stop - rows.start
    q = s["q"][rows, kv.start * g: kv.stop * g].float().unflatten(1, (-1, g)).permute(1, 2, 0, 3)
    k, v = (s[t][rows, kv].float().transpose(0, 1) for t in "kv")
    t = (q.reshape(q.shape[0], g * n, -1) @ k.transpose(1, 2) * s["scale"]).view(-1, g, n, n)
    if c["causal"]:
        i = torch.arange(n, device=t.device)
        t = t.masked_fill(i[None, :] > i[:, None], -math.inf)
    return t, q, k, v


def _plain_fwd(s):
    c = s["c"]
    g = c["Hq"] // c["Hkv"]
    o, lse = torch.zeros_like(s["o"]), torch.zeros_like(s["lse"])
    for rows, kv in _parts(s):
        t, _, _, v = _scores(s, rows, kv)
        top = t.amax(-1, keepdim=True)
        p = torch.exp(t - top)
        l = p.sum(-1, keepdim=True)
        heads = slice(kv.start * g, kv.stop * g)
        out = (p.flatten(1, 2) @ v).view(*p.shape[:3], -1) / l
        o[rows, heads] = out.flatten(0, 1).transpose(0, 1).to(torch.bfloat16)
        lse[heads, rows] = (torch.log(l) + top).flatten(0, 1)[..., 0]
    return o, lse


def _plain_bwd(s):
    c = s["c"]
    g = c["Hq"] // c["Hkv"]
    grad = torch.zeros_like(s["dqkv"])
    dq, dk, dv = grad.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
    for rows, kv in _parts(s):
        t, q, k, v = _scores(s, rows, kv)
        heads = slice(kv.start * g, kv.stop * g)
        do, o = (s[x][rows, heads].float().unflatten(1, (-1, g)).permute(1, 2, 0, 3) for x in ("do", "o"))
        p = torch.exp(t - s["lse"][heads, rows].unflatten(0, (-1, g))[..., None]).flatten(1, 2)
        D = (do * o).sum(-1, keepdim=True).flatten(1, 2)
        do, q = do.flatten(1, 2), q.flatten(1, 2)
        ds = p * (do @ v.transpose(1, 2) - D) * s["scale"]
        dq[rows, heads] = (ds @ k).unflatten(1, (g, -1)).flatten(0, 1).transpose(0, 1).to(torch.bfloat16)
        dk[rows, kv] = (ds.transpose(1, 2) @ q).transpose(0, 1).to(torch.bfloat16)
        dv[rows, kv] = (p.transpose(1, 2) @ do).transpose(0, 1).to(torch.bfloat16)
    return grad


_PLAIN = {"axes_fwd": _plain_axes_fwd, "axes_bwd": _plain_axes_bwd, "packed_fwd": _plain_fwd, "packed_bwd": _plain_bwd}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(c, seed):
    global own
    was, own = own, False
    try:
        # 64-bit products run at about a TFLOP/s, over the whole square of scores
        if c["op"].startswith("packed"):
            products = 2 if c["op"] == "packed_fwd" else 5
            if 2 * products * c["d"] * c["Hq"] * sum(n * n for n in _lens(c)) > 1e13:
                return None
        s = prepare(c, seed)
    finally:
        own = was
    return {"axes_fwd": _exact_axes, "axes_bwd": _exact_axes, "packed_fwd": _exact_fwd,
            "packed_bwd": _exact_bwd}[c["op"]](s)


def _exact_axes(s):
    """The rotation as a product of complex numbers; the backward pass by its Jacobian."""
    c, f64 = s["c"], torch.float64
    axis = s["axes"]
    rot = 2 * len(axis)
    phase = torch.complex(s["cos"].to(f64), s["sin"].to(f64))
    phase = torch.stack([phase[s["pos"][a].long(), i] for i, a in enumerate(axis)], -1)[:, None]  # [B, 1, N, rot / 2]

    def turn(x, ph):
        head, rest = x[..., :rot], x[..., rot:]
        if c["interleaved"]:
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * ph
            return torch.cat((torch.view_as_real(z).flatten(-2), rest), -1)
        z = torch.complex(head[..., : rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * ph
        return torch.cat((z.real, z.imag, rest), -1)

    def rms(x):
        return (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt()

    if c["op"] == "axes_fwd":
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


def _rows64(s):
    """(first row, sequence's length, query head, K/V head) of every piece in turn."""
    c, at = s["c"], 0
    for n in s["lens"]:
        for h in range(c["Hq"] if n else 0):
            yield slice(at, at + n), h, h // (c["Hq"] // c["Hkv"])
        at += n


def _scores64(s, rows, h, kv):
    t = torch.einsum("nd,ld->nl", s["q"][rows, h].double(), s["k"][rows, kv].double()) * s["scale"]
    if s["c"]["causal"]:
        t = t + torch.full_like(t, -math.inf).triu_(1)
    return t


def _exact_fwd(s):
    o, lse = s["o"].double(), s["lse"].double()
    for rows, h, kv in _rows64(s):
        t = _scores64(s, rows, h, kv)
        lse[h, rows] = torch.logsumexp(t, -1)
        o[rows, h] = torch.softmax(t, -1) @ s["v"][rows, kv].double()
    return o, lse


def _exact_bwd(s):
    """The gradients for the outputs that the call is given: the softmax from its stored logarithms, the
    row sums from its stored outputs."""
    c = s["c"]
    Hq, Hkv = c["Hq"], c["Hkv"]
    grad = torch.zeros(s["qkv"].shape, dtype=torch.float64, device=s["qkv"].device)
    for rows, h, kv in _rows64(s):
        q, k, v = s["q"][rows, h].double(), s["k"][rows, kv].double(), s["v"][rows, kv].double()
        do = s["do"][rows, h].double()
        p = torch.exp(_scores64(s, rows, h, kv) - s["lse"][h, rows].double()[:, None])
        ds = p * (torch.einsum("nd,ld->nl", do, v) - torch.einsum("nd,nd->n", do, s["o"][rows, h].double())[:, None])
        grad[rows, h] = ds @ k * s["scale"]
        grad[rows, Hq + kv] += torch.einsum("nl,nd->ld", ds, q) * s["scale"]
        grad[rows, Hq + Hkv + kv] += torch.einsum("nl,nd->ld", p, do)
    return grad
