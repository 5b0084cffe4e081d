"""Cases, plain forms and exact values of the serving operators around the
paged FP4 cache:

  append   csa2_append_kv_rope: new tokens' latents (and indexer keys) are
           rotated by their position, quantised (E2M1 with one E4M3 scale per
           16 channels; E4M3 with one binary32 scale per row) and written to
           their slots of the paged cache.
  rope     csa2_rope_rows: the same rotation of query rows.
  attn     csa2_group_attn: every query token of a group attends to all the
           cache entries of its group. One group with a batch's query tokens
           is attention over a prefix that the batch shares, joined with each
           token's own part (its normalised result and log-sum-exp over its
           own keys); one group per sequence is cross attention to states of
           another length.

`own` picks the framework's kernels; otherwise `run` computes in plain torch.
"""
import math
import random

import torch

own = False

HEADS, DIM, IDX_DIM, PAGE, GROUP = 16, 576, 64, 64, 16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E2M1_MID = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
SCALE = 1.0 / math.sqrt(DIM)
ROPE_BASE = 10000.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 sequences in a long context: one token each, indexer keys too
        dict(name="append_decode_b64", op="append", tokens=64, rope=64, interleaved=True, keys=True, far=131072,
             bulk=False, pad=False, stride=576),
        # a draft verified by 32 sequences, 4 tokens each, some padded away, latents inside wider rows
        dict(name="append_verify_b32_sq4", op="append", tokens=128, rope=64, interleaved=False, keys=True, far=32768,
             bulk=False, pad=True, stride=640),
        # a whole 128K prompt
        dict(name="append_prompt_128k", op="append", tokens=131072, rope=64, interleaved=True, keys=True, far=1048576,
             bulk=True, pad=False, stride=576),
        # the decode step's attention queries
        dict(name="rope_query_b64", op="rope", tokens=64, heads=16, dim=576, rope=64, interleaved=True, far=131072),
        # a prompt chunk's indexer queries, far into a context
        dict(name="rope_index_query_16k", op="rope", tokens=16384, heads=4, dim=64, rope=64, interleaved=False,
             far=1048576),
        # one sequence's token over a 4K prefix: latency
        dict(name="prefix_b1_t4k", op="attn", groups=1, tokens=1, len=4096, ragged=False, own_part=True, shape=1),
        # a batch of 64 behind one 32K prompt
        dict(name="prefix_b64_t32k", op="attn", groups=1, tokens=64, len=32768, ragged=False, own_part=True, shape=2),
        # 32 sequences verifying 4 tokens each behind one 16K prompt
        dict(name="prefix_b32_sq4_t16k", op="attn", groups=1, tokens=128, len=16384, ragged=False, own_part=True,
             shape=3),
        # several prompts of uneven length and popularity in one batch, one of them empty
        dict(name="prefix_groups_ragged", op="attn", groups=6, tokens=75, len=12345, ragged=True, own_part=True,
             shape=4),
        # four sequences over a 1M-token context
        dict(name="prefix_b4_t1m", op="attn", groups=1, tokens=4, len=1048576, ragged=False, own_part=False, shape=5),
        # cross attention: 64 decoder tokens of each of 8 sequences over their encoder's states, ragged lengths
        dict(name="cross_b8_l64", op="attn", groups=8, tokens=512, len=4096, ragged=True, own_part=False, shape=6),
        # cross attention of one decode step: one token of each of 64 sequences
        dict(name="cross_b64_l1", op="attn", groups=64, tokens=64, len=4096, ragged=False, own_part=False, shape=7),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "rope", "attn", "attn"))
    if op == "append":
        n = _log_int(rng, 1, 100000)
        return dict(op=op, tokens=n, rope=rng.choice((16, 32, 64, 96)), interleaved=rng.random() < 0.5,
                    keys=rng.random() < 0.7, far=_log_int(rng, 2 * n + 8, 1 << 20), bulk=rng.random() < 0.5,
                    pad=rng.random() < 0.3, stride=rng.choice((576, 584, 640, 1152)))
    if op == "rope":
        heads, dim = rng.choice(((16, 576), (4, 64), (1, 576)))
        return dict(op=op, tokens=_log_int(rng, 1, 4096), heads=heads, dim=dim, rope=rng.choice((16, 32, 64)),
                    interleaved=rng.random() < 0.5, far=_log_int(rng, 64, 1 << 20))
    groups = rng.choice((1, 1, 2, 5, 17))
    tokens = _log_int(rng, groups, 256)
    most = min(131072, (64 * 32768) // tokens)
    return dict(op=op, groups=groups, tokens=tokens, len=_log_int(rng, 1, most), ragged=rng.random() < 0.6,
                own_part=rng.random() < 0.6, shape=rng.randrange(1 << 20))


def _layout(case):
    """Query tokens and cache entries of each group."""
    G, N, T = case["groups"], case["tokens"], case["len"]
    if not case["ragged"]:
        n = [N // G + (g < N % G) for g in range(G)]
        return n, [T] * G
    r = random.Random(case["shape"])
    cuts = sorted(r.randrange(N + 1) for _ in range(G - 1))
    n = [b - a for a, b in zip([0] + cuts, cuts + [N])]
    t = [r.randrange(T + 1) for _ in range(G)]
    t[r.randrange(G)] = T
    if G > 2:
        t[(t.index(T) + 1) % G] = 0
    return n, t


def work(case):
    n = case["tokens"]
    if case["op"] == "append":
        kept = n - n // 8 if case["pad"] else n
        per = DIM * 2 + 8 + 324 + ((IDX_DIM * 2 + 68) if case["keys"] else 0)
        return {"bytes": kept * per, "flops": kept * (DIM * 4 + 6 * case["rope"])}
    if case["op"] == "rope":
        return {"bytes": n * (4 + 4 * case["heads"] * case["dim"]), "flops": n * case["heads"] * case["rope"] * 3}
    rows, lens = _layout(case)
    bytes_ = sum(324 * t for t in lens) + n * (HEADS * DIM * 4 + HEADS * 4)
    if case["own_part"]:
        bytes_ += n * HEADS * (DIM + 1) * 4
    return {"bytes": bytes_, "flops": sum(r * HEADS * t * 4 * DIM for r, t in zip(rows, lens))}


# ------------------------------------------------------------------ inputs
def _latents(n, g, dev):
    """Latent rows with a few large channels."""
    x = torch.randn(n, DIM, generator=g, device=dev)
    big = torch.randperm(DIM, generator=g, device=dev)[:6]
    x[:, big] *= 8.0
    return x


def _pages(lens):
    return [-(-t // PAGE) for t in lens]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    n = case["tokens"]
    s = {"case": case}
    if case["op"] != "attn":
        R = case["rope"]
        s["inv_freq"] = (ROPE_BASE ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).to(torch.float32).to(dev)
        if case["op"] == "append" and case["bulk"]:
            first = int(torch.randint(0, max(1, case["far"] - n), (1,), generator=g, device=dev))
            s["pos"] = torch.arange(first, first + n, device=dev, dtype=torch.int32)
        else:
            s["pos"] = torch.randint(0, case["far"], (n,), generator=g, device=dev, dtype=torch.int32)
    if case["op"] == "rope":
        s["x"] = torch.randn(n, case["heads"], case["dim"], generator=g, device=dev).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["x"])
        if own:
            from compressed_sparse_attention_quant_b200 import lib
            s["rope"] = lib.Rope(s["inv_freq"], case["dim"] - R, case["interleaved"])
        return s
    if case["op"] == "append":
        wide = torch.zeros(n, case["stride"], device=dev, dtype=torch.bfloat16)
        wide[:, :DIM] = _latents(n, g, dev).to(torch.bfloat16)
        s["x"] = wide[:, :DIM]
        s["kidx"] = torch.randn(n, IDX_DIM, generator=g, device=dev).to(torch.bfloat16) if case["keys"] else None
        pages = -(-n // PAGE) + 1
        s["pages"] = pages
        if case["bulk"]:
            perm = torch.randperm(pages, generator=g, device=dev)
            t = torch.arange(n, device=dev)
            s["slots"] = (perm[t // PAGE] * PAGE + t % PAGE).to(torch.int32)
        else:
            s["slots"] = torch.randperm(pages * PAGE, generator=g, device=dev)[:n].to(torch.int32)
        if case["pad"]:
            s["slots"][torch.randperm(n, generator=g, device=dev)[: n // 8]] = -1
        s["table"] = _pair_table(dev)
        if own:
            from compressed_sparse_attention_quant_b200 import lib
            c = s["cache"] = lib.PagedCache(pages, dev)
            s["held"] = [c.kv_fp4, c.kv_scale, c.kidx, c.kidx_scale]
            s["rope"] = lib.Rope(s["inv_freq"], DIM - case["rope"], case["interleaved"])
            R = min(case["rope"], IDX_DIM)
            s["kidx_rope"] = lib.Rope(s["inv_freq"][: R // 2], 0, case["interleaved"])
        else:
            u8 = dict(dtype=torch.uint8, device=dev)
            s["held"] = [torch.zeros(pages, PAGE, DIM // 2, **u8), torch.zeros(pages, PAGE, DIM // GROUP, **u8),
                         torch.zeros(pages, PAGE * IDX_DIM, **u8), torch.zeros(pages, PAGE, device=dev)]
        return s
    # attention: a cache of quantised latents, its pages in random order
    rows, lens = _layout(case)
    per = _pages(lens)
    width, total = max(max(per), 1), max(sum(per), 1)
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device=dev)
    at = 0
    for i, p in enumerate(per):
        table[i, :p] = perm[at: at + p]
        at += p
    kv = torch.zeros(total * PAGE, DIM // 2, dtype=torch.uint8, device=dev)
    sc = torch.zeros(total * PAGE, DIM // GROUP, dtype=torch.uint8, device=dev)
    step = 65536
    for a in range(0, total * PAGE, step):
        b = min(total * PAGE, a + step)
        kv[a:b], sc[a:b] = _fp4(_latents(b - a, g, dev).to(torch.bfloat16).float())
    s["kv"], s["sc"] = kv.view(total, PAGE, DIM // 2), sc.view(total, PAGE, DIM // GROUP)
    s["table_pages"] = table
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["offsets"] = torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32, device=dev)
    s["q"] = torch.randn(n, HEADS, DIM, generator=g, device=dev).to(torch.bfloat16)
    s["o_own"] = s["lse_own"] = None
    if case["own_part"]:
        # what a token's own keys (a window and its selected entries) gave it
        s["o_own"] = torch.randn(n, HEADS, DIM, generator=g, device=dev) * 0.2
        s["lse_own"] = 7.0 + torch.randn(n, HEADS, generator=g, device=dev) * 0.3
    if own:
        from compressed_sparse_attention_quant_b200 import lib
        c = s["cache"] = lib.PagedCache(total, dev)
        c.kv_fp4.copy_(s["kv"])
        c.kv_scale.copy_(s["sc"])
        s["ws"] = lib.workspace(lib.group_attn_workspace_bytes(n, len(lens)), dev)
        s["out"] = torch.empty(n, HEADS, DIM, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(n, HEADS, dtype=torch.float32, device=dev)
    else:
        width_rows = max(max(rows), 1)
        # row r of group i is token offsets[i] + r; rows past a group's tokens are masked
        r = torch.arange(width_rows, device=dev)
        s["row_ok"] = r[None] < torch.tensor(rows, device=dev)[:, None]
        s["row_tok"] = (s["offsets"][:-1, None] + r[None]).clamp(max=n - 1).long()
    return s


# ------------------------------------------------------------------ plain forms
def _pair_table(dev):
    """The four E2M1 values of two packed bytes, as four bf16 in one 64-bit word, by their 16 bits."""
    code = torch.arange(65536, device=dev)
    nib = torch.stack([(code >> (4 * i)) & 15 for i in range(4)], 1)
    val = torch.tensor(E2M1, device=dev)[nib & 7] * torch.where(nib >= 8, -1.0, 1.0)
    return val.to(torch.bfloat16).contiguous().view(torch.int64).view(-1)


def _held_values(s):
    """The cache's contents as the values they stand for."""
    kv, sc, ki, sg = s["held"]
    vals = s["table"][kv.view(torch.uint16).int()].view(torch.bfloat16)
    if s["kidx"] is None:
        return {"codes": vals, "scales": sc.view(torch.float8_e4m3fn)}
    return {"codes": vals, "scales": sc.view(torch.float8_e4m3fn), "keys": ki.view(torch.float8_e4m3fn), "sigma": sg}


def _rotate(x, pos, inv_freq, offset, interleaved):
    """Rotates channels offset .. offset + 2 len(inv_freq) of x [n, ..., D] by angle pos * inv_freq: angles and
    products in 64 bits (positions are far), rounded to binary32 and then to bf16."""
    half = inv_freq.numel()
    R = 2 * half
    ang = pos.double()[:, None] * inv_freq.double()
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (half,)
    c, sn = torch.cos(ang).view(shape), torch.sin(ang).view(shape)
    part = x[..., offset:offset + R].double()
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :half], part[..., half:])
    ra, rb = a * c - b * sn, a * sn + b * c
    rot = torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1)
    out = x.clone()
    out[..., offset:offset + R] = rot.float().to(torch.bfloat16)
    return out


def _fp4(x):
    """Packed E2M1 codes and E4M3 scale bytes of fp32 rows [n, 576]."""
    grp = x.view(-1, DIM // GROUP, GROUP)
    mag = grp.abs()
    scale = (mag.amax(-1).double() / 6.0).float().clamp(max=448.0).to(torch.float8_e4m3fn)     # the rounded quotient
    s = scale.float()[..., None]
    code = torch.zeros_like(mag, dtype=torch.uint8)
    for i, m in enumerate(E2M1_MID):       # ties go to the even code
        code += (mag > s * m) if i % 2 == 0 else (mag >= s * m)
    code = torch.where(s > 0, code, torch.zeros_like(code))
    code = torch.where((grp < 0) & (code > 0), code | 8, code).view(-1, DIM)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale.view(torch.uint8)


def _fp8_rows(x):
    """E4M3 codes and binary32 scales of bf16 rows [n, 64]: the exact quotient rounded once, so in 64 bits."""
    sigma = (x.double().abs().amax(-1) / 448.0).float()
    q = torch.where(sigma[:, None] > 0, x.double() / sigma.double()[:, None], torch.zeros((), device=x.device).double())
    _, e = torch.frexp(q)
    ulp = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    v = (torch.round(q / ulp) * ulp).clamp(-448.0, 448.0)
    v = torch.where(v == 0, torch.zeros_like(v), v)
    return v.float().to(torch.float8_e4m3fn).view(torch.uint8), sigma


def _append_plain(s):
    case, pos, slots = s["case"], s["pos"], s["slots"].long()
    kv, sc, ki, sg = s["held"]
    keep = slots >= 0
    slots = slots[keep] if case["pad"] else slots
    take = (lambda t: t[keep]) if case["pad"] else (lambda t: t)
    pos = take(pos)
    codes, scale = _fp4(_rotate(take(s["x"]), pos, s["inv_freq"], DIM - case["rope"], case["interleaved"]).float())
    kv.view(-1, DIM // 2)[slots] = codes
    sc.view(-1, DIM // GROUP)[slots] = scale
    if s["kidx"] is not None:
        half = min(case["rope"], IDX_DIM) // 2
        k8, sigma = _fp8_rows(_rotate(take(s["kidx"]), pos, s["inv_freq"][:half], 0, case["interleaved"]))
        # a page's keys lie in 8 x 16-byte blocks: [t / 8][c / 16][t % 8][c % 16]
        blocks = ki.view(-1, 8, 4, 8, 16)
        t = slots % PAGE
        blocks[slots // PAGE, t // 8, :, t % 8] = k8.view(-1, 4, 16)
        sg.view(-1)[slots] = sigma
    return _held_values(s)


def _dequant(kv, sc, dtype):
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=kv.device, dtype=dtype)
    codes = torch.stack((kv & 15, kv >> 4), -1).flatten(-2).int()
    return (v[codes].unflatten(-1, (DIM // GROUP, GROUP)) *
            sc.view(torch.float8_e4m3fn).to(dtype)[..., None]).flatten(-2)


def _attn_plain(s):
    """All groups at once, padded to the longest: rows [G, L * 16, 576] against keys [G, T, 576]."""
    table, lens, q = s["table_pages"], s["lens"], s["q"]
    G, W = table.shape
    keys = _dequant(s["kv"][table.long()].view(G, W * PAGE, -1), s["sc"][table.long()].view(G, W * PAGE, -1),
                    torch.float32)
    rows = q.float()[s["row_tok"]].view(G, -1, DIM)
    sc = torch.bmm(rows, keys.transpose(1, 2)).mul_(SCALE)
    dead = torch.arange(W * PAGE, device=q.device)[None] >= lens[:, None]
    sc.masked_fill_(dead[:, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    keys = torch.where(dead[..., None], torch.zeros((), device=q.device), keys)
    o = torch.bmm(p, keys) / l.clamp(min=1e-30)
    lse = torch.where(l > 0, m + torch.log(l.clamp(min=1e-30)), torch.full_like(l, -math.inf))
    ok = s["row_ok"]
    out = torch.zeros(q.shape, device=q.device)
    lse_out = torch.full(q.shape[:2], -math.inf, device=q.device)
    out[s["row_tok"][ok]] = o.view(G, -1, HEADS, DIM)[ok]
    lse_out[s["row_tok"][ok]] = lse.view(G, -1, HEADS)[ok]
    if s["o_own"] is not None:
        both = torch.logaddexp(lse_out, s["lse_own"])
        out = out * (lse_out - both).exp()[..., None] + s["o_own"] * (s["lse_own"] - both).exp()[..., None]
        lse_out = both
    return {"out": out.to(torch.bfloat16), "lse": lse_out}


def run(state):
    s = state
    case = s["case"]
    if own:
        from compressed_sparse_attention_quant_b200 import lib
        if case["op"] == "append":
            lib.append_kv_rope(s["x"], s["pos"], s["slots"], s["cache"], s["rope"], s["kidx"],
                               s["kidx_rope"] if case["keys"] else None)
            return _held_values(s)
        if case["op"] == "rope":
            return lib.rope_rows(s["x"], s["pos"], s["rope"], out=s["out"])
        out, lse = lib.group_attn(s["q"], s["cache"], s["table_pages"], s["lens"], s["offsets"], SCALE,
                                  o_own=s["o_own"], lse_own=s["lse_own"], out=s["out"], lse=s["lse"], ws=s["ws"])
        return {"out": out, "lse": lse}
    if case["op"] == "append":
        return _append_plain(s)
    if case["op"] == "rope":
        return _rotate(s["x"], s["pos"], s["inv_freq"], case["dim"] - case["rope"], case["interleaved"])
    return _attn_plain(s)


# ------------------------------------------------------------------ exact values
def _exact_rotate(x, pos, freq, first, interleaved):
    """One complex product per pair, in 64 bits, rounded to bf16 by way of binary32."""
    half = freq.numel()
    i = torch.arange(half, device=x.device)
    ia, ib = (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + half + i)
    turn = torch.polar(torch.ones((), device=x.device, dtype=torch.float64), pos.double()[:, None] * freq.double()[None])
    while turn.dim() < x.dim():
        turn = turn.unsqueeze(1)
    z = torch.complex(x[..., ia].double(), x[..., ib].double()) * turn
    y = x.double().clone()
    y[..., ia] = z.real.float().to(torch.bfloat16).double()
    y[..., ib] = z.imag.float().to(torch.bfloat16).double()
    return y


def _nearest(v, table):
    """Index of the entry of an ascending table that is nearest to v >= 0; a tie goes to the even index."""
    mid = (table[1:] + table[:-1]) / 2
    lo, hi = torch.searchsorted(mid, v, right=False), torch.searchsorted(mid, v, right=True)
    return torch.where(lo % 2 == 0, lo, hi)


def _exact_append(s):
    case = s["case"]
    dev = s["x"].device
    e4m3 = torch.arange(127, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    e2m1 = torch.tensor(E2M1, device=dev, dtype=torch.float64)
    pages = s["pages"]
    codes = torch.zeros(pages * PAGE, DIM, device=dev, dtype=torch.float64)
    scales = torch.zeros(pages * PAGE, DIM // GROUP, device=dev, dtype=torch.float64)
    keys = torch.zeros(pages, 8, 4, 8, 16, device=dev, dtype=torch.float64)
    sigma = torch.zeros(pages * PAGE, device=dev, dtype=torch.float64)
    step = 16384
    for a in range(0, case["tokens"], step):
        sl = s["slots"][a:a + step].long()
        ok = sl >= 0
        sl, pos = sl[ok], s["pos"][a:a + step][ok]
        y = _exact_rotate(s["x"][a:a + step][ok], pos, s["inv_freq"], DIM - case["rope"], case["interleaved"])
        y = y.view(-1, DIM // GROUP, GROUP)
        sc = e4m3[_nearest(y.abs().amax(-1) / 6, e4m3)]
        v = e2m1[_nearest(torch.where(sc[..., None] > 0, y.abs() / sc[..., None], torch.zeros_like(y)), e2m1)]
        codes[sl] = (v * torch.sign(y)).view(-1, DIM)
        scales[sl] = sc
        if case["keys"]:
            half = min(case["rope"], IDX_DIM) // 2
            y = _exact_rotate(s["kidx"][a:a + step][ok], pos, s["inv_freq"][:half], 0, case["interleaved"])
            sg = (y.abs().amax(-1) / 448).float().double()
            v = e4m3[_nearest(y.abs() / sg[:, None], e4m3)] * torch.sign(y)
            t = sl % PAGE
            keys[sl // PAGE, t // 8, :, t % 8] = v.view(-1, 4, 16)
            sigma[sl] = sg
    got = {"codes": codes.view(pages, PAGE, DIM), "scales": scales.view(pages, PAGE, -1)}
    if case["keys"]:
        got |= {"keys": keys.view(pages, -1), "sigma": sigma.view(pages, PAGE)}
    return got


def _exact_attn(s):
    """Group by group and block of keys by block, one running maximum and sum per row."""
    q, dev = s["q"], s["q"].device
    out = torch.zeros(q.shape, device=dev, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, device=dev, dtype=torch.float64)
    lens, offs = s["lens"].tolist(), s["offsets"].tolist()
    for g, T in enumerate(lens):
        a, b = offs[g], offs[g + 1]
        if a == b:
            continue
        rows = q[a:b].double().reshape(-1, DIM)
        m = torch.full((rows.shape[0], 1), -math.inf, device=dev, dtype=torch.float64)
        l = torch.zeros_like(m)
        acc = torch.zeros_like(rows)
        for t0 in range(0, T, 32768):
            t = torch.arange(t0, min(T, t0 + 32768), device=dev)
            page = s["table_pages"][g].long()[t // PAGE]
            k = _dequant(s["kv"][page, t % PAGE], s["sc"][page, t % PAGE], torch.float64)
            sc = rows @ k.t() * SCALE
            m_new = torch.maximum(m, sc.amax(-1, keepdim=True))
            w, old = torch.exp(sc - m_new), torch.exp(m - m_new)
            l, acc, m = l * old + w.sum(-1, keepdim=True), acc * old + w @ k, m_new
        if s["o_own"] is not None:
            lo = s["lse_own"][a:b].double().reshape(-1, 1)
            m_new = torch.maximum(m, lo)
            old, w = torch.exp(m - m_new), torch.exp(lo - m_new)
            l, acc = l * old + w, acc * old + w * s["o_own"][a:b].double().reshape(-1, DIM)
            m = m_new
        some = l > 0
        out[a:b] = torch.where(some, acc / l, torch.zeros_like(acc)).view(b - a, HEADS, DIM)
        lse[a:b] = torch.where(some, m + torch.log(l), torch.full_like(l, -math.inf)).view(b - a, HEADS)
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "rope":
        return _exact_rotate(s["x"], s["pos"], s["inv_freq"], case["dim"] - case["rope"], case["interleaved"])
    return _exact_attn(s)
