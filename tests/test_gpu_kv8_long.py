"""GPU parity of fa_fwd_kv8 on calls so long that both of its kernels reach their
steady state: every ring wraps many times, a run crosses heads and sequences,
page batches and tables are refilled. Sampled heads, all of their rows, against
float64 on the device from the same codes.

Tolerances. With p the exact weights and n keys, O = sum p_j v_j / 1:
  - the output's rounding, 2^-8 |O|;
  - each weight is off by a factor 1 + e_j, |e_j| <= 2^-11 (fp16) + 2^-20 (exp2 and
    its factors) + 2 delta, where delta bounds a score's error (below). The signs
    of V are drawn independently of everything the e_j depend on (queries, keys,
    |V|), so sum e_j p_j v_j passes t sqrt(sum (max|e| p_j v_j)^2) with probability
    2 exp(-t^2 / 2) at most (Hoeffding); t = 8 leaves 10^-13 an element;
  - fp16's smallest step, 2^-24 of a row's largest weight times its page's scale,
    likewise: t 2^-24 max(p) (S / s) sqrt(sum v_j^2) with S, s the largest and
    smallest value scale (all pages hold values of one distribution);
  - fp32 sums: c additions in a chain at most, of 2^-23 each (the tensor core may
    cut instead of round): c 2^-23 sum p_j |v_j|;
  - the sum of the weights, off by the bound of L: |O| times it.
A score is a sum of d exact products in fp32 (two units of 2^-23 for each of d / 16
steps, four for its scaling) of query values exact or within e max|q|: e = 2^-21 up
to 16 rows per K/V head (8 at d = 256), two e4m3 pieces summed with a factor of 2^4
between them, and 2^-17 above, where they are not:
  delta = scale max_j ((d/16 + 4) 2^-22 sum |q k_j| + e max|q| sum |k_j|)
  |L - L_ref| <= delta + 2^-20 + c_l 2^-24 + 2^-21 |L_ref|, c_l additions in a chain.
"""

import math

import pytest

from attn_inputs import BASE_SEED

pytestmark = pytest.mark.gpu

T = 8.0
ROWS_FEW = {64: 16, 128: 16, 256: 8}  # most rows per K/V head of the kernel that streams key steps
WARPS = {64: 12, 128: 8, 256: 4}      # of a CTA of it


def make(B, Hkv, d, page, lens, seed):
    """Codes and scales of random tokens, pages in random order, unwritten ones full of any bytes."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    mp = -(-max(lens) // page)
    pages = B * mp + 3
    table = torch.randperm(pages, generator=gen, device="cuda")[:B * mp].view(B, mp).to(torch.int32)
    code, scale = [], []
    for _ in range(2):
        x = torch.randn(pages, Hkv, page, d, generator=gen, device="cuda")
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448)))
        code.append((x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8))
        scale.append(s)
    held = torch.zeros(pages, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        used = -(-n // page)
        held[table[b, :used].long()] = True
        if n % page:  # behind the last token
            code[0][table[b, used - 1].long(), :, n % page:] = 0x7F
            code[1][table[b, used - 1].long(), :, n % page:] = 0xFF
    for i in range(2):
        code[i][~held] = 0x7F
        scale[i][~held] = float("nan")
    for b, n in enumerate(lens):
        table[b, -(-n // page):] = -1
    return gen, code, scale, table


def rows_of(code, scale, table, b, h, n):
    import torch
    page = code.shape[2]
    p = table[b, :-(-n // page)].long()
    x = code[p, h].view(torch.float8_e4m3fn).double() * scale[p, h].double()[:, None, None]
    return x.flatten(0, 1)[:n]


def check(Hq, Hkv, Nq, d, page, lens, causal, seed, least):
    """least: key tiles a CTA takes (many rows) or key steps a warp takes (few rows), at least."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, g = len(lens), Hq // Hkv
    few = g * Nq <= ROWS_FEW[d]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if few:
        per = 4 if d == 256 or g * Nq <= 4 else 8
        taken = sum(-(-n // 32) for n in lens) * Hkv * -(-g * Nq // per) / (sms * WARPS[d])
        chain = math.ceil(taken) * 2 + 4 * sms  # MMAs of a run, then the parts of a row
        chain_l = math.ceil(taken) * 4 + 8 + 4 * sms
    else:
        block = 128 if d == 256 else 256
        taken = sum(-(-n // 128) for n in lens) * Hkv * -(-g * Nq // block) / sms
        chain = math.ceil(taken) * 8 + sms
        chain_l = math.ceil(taken) * 72 + sms  # 64 pairs and 8 groups a tile
    assert taken >= least, taken
    gen, code, scale, table = make(B, Hkv, d, page, lens, seed)
    q = torch.randn(B, Hq, Nq, d, generator=gen, device="cuda").bfloat16()
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.full((fa.fa_fwd_kv8_workspace_size(B, Hq, Hkv, Nq, d),), 255, dtype=torch.uint8, device="cuda")
    c = 1 / math.sqrt(d)

    def run():
        o, lse = torch.full_like(q, 7.0), torch.full((B, Hq, Nq), 7.0, device="cuda")
        fa.fa_fwd_kv8(q, *code, *scale, table, lens_d, o, lse, causal, c, None, ws)
        return o, lse

    o, lse = run()
    again = run()
    assert fa.fa_get_device_status() == 0
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    e_q = 2.0 ** -21 if few else 2.0 ** -17
    for b, h in {(0, 0), (B - 1, Hkv - 1), (B // 2, Hkv // 2), (B // 3, 1 % Hkv), (2 * B // 3, Hkv - 1)}:
        n = lens[b]
        k, v = (rows_of(code[i], scale[i], table, b, h, n) for i in range(2))
        s_v = scale[1][table[b, :-(-n // page)].long(), h]
        spread = float(s_v.max() / s_v.min())
        qr = q[b, h * g:(h + 1) * g].double()  # [g, Nq, d]
        pos = torch.arange(Nq, device="cuda") + n - Nq
        see = torch.arange(n, device="cuda")[None, :] <= (pos[:, None] if causal else n)
        for r in range(g):
            t = (c * (qr[r] @ k.T)).masked_fill(~see, -math.inf)
            ref_l = torch.logsumexp(t, 1)
            w = torch.exp(t - ref_l[:, None])
            ref = w @ v
            A, A2 = w @ v.abs(), torch.sqrt((w * w) @ (v * v))
            mag = (d / 16 + 4) * 2.0 ** -22 * (qr[r].abs() @ k.abs().T)
            mag += e_q * qr[r].abs().amax(1, keepdim=True) * k.abs().sum(1)[None, :]
            delta = c * mag.masked_fill(~see, 0).amax(1)
            tol_l = delta + 2.0 ** -20 + chain_l * 2.0 ** -24 + 2.0 ** -21 * ref_l.abs()
            err_l = (lse[b, h * g + r].double() - ref_l).abs()
            assert (err_l <= tol_l).all(), (b, h, r, float(err_l.max()), float(tol_l.min()))
            tol = 2.0 ** -8 * ref.abs() + T * (2.0 ** -11 + 2.0 ** -20 + 2 * delta[:, None]) * A2
            tol += T * 2.0 ** -24 * spread * w.amax(1, keepdim=True) * torch.sqrt(see.double() @ (v * v))
            tol += chain * 2.0 ** -23 * A + tol_l[:, None] * ref.abs()
            err = (o[b, h * g + r].double() - ref).abs()
            assert (err <= tol).all(), (b, h, r, float(err.max()), float((err - tol).max()))


def ragged(B, longest, seed):
    import random
    rng = random.Random(seed)
    return [longest] + [rng.randint(longest // 2, longest) for _ in range(B - 2)] + [rng.randint(1, 300)]


# keys of the longest of 10 sequences with 8 heads, so that a warp takes 40 steps or more
FEW = {64: 47000, 128: 30000, 256: 15000}


@pytest.mark.parametrize("d,page,g,Nq", [(d, *x) for d in (64, 128, 256) for x in ((16, 1, 1), (128, 4, 1), (64, 8, 1), (32, 3, 2))] +
                         [(64, 16, 4, 4), (128, 16, 4, 4)])
def test_few_rows_a_head(d, page, g, Nq):
    # 40 steps a warp: the ring of three or four stages wraps ten times, the page batches of 16 steps twice
    lens = [max(n, Nq) for n in ragged(10, FEW[d], d + page)]
    check(8 * g, 8, Nq, d, page, lens, True, BASE_SEED + d + g, 40)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page,g,Nq", [(16, 4, 5), (128, 8, 10), (64, 2, 64), (32, 1, 100)])
def test_one_tile_of_rows(d, page, g, Nq, causal):
    # 20, 80, 128 and 100 rows: at d = 64 and 128 the slots take every other key tile each
    lens = [max(n, Nq) for n in ragged(8, 8000, d + page + Nq)]
    check(8 * g, 8, Nq, d, page, lens, causal, BASE_SEED + d + Nq, 15)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page,g,Nq", [(16, 3, 100), (128, 1, 200), (64, 5, 77)])
def test_blocks_of_two_tiles_of_rows(d, page, g, Nq, causal):
    # 300, 200 and 385 rows: one or two blocks of two tiles (d = 256: of one)
    lens = [max(n, Nq) for n in ragged(6, 7000, d + page + Nq)]
    check(8 * g, 8, Nq, d, page, lens, causal, BASE_SEED + d + Nq, 8)


@pytest.mark.parametrize("d", [64, 128])
def test_one_long_sequence_in_one_tile_of_rows(d):
    # one head: each CTA has one part of the same block, all of 25 key tiles
    check(8, 1, 4, d, 64, [152 * 25 * 128 + 77], True, BASE_SEED + d, 25)
