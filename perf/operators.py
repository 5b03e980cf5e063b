"""The serving and training operators around Parallax attention, as cases to measure.

    page_plan       page table, slot map and positions of one step, from request lengths
    norm_rope       RMS norm of every query, probe and key head with the position rotation, and its backward
    append_q4       keys and values into the 4-bit paged cache, and read back
    decode_q4       Parallax decode over the 4-bit cache

``run`` is the plain form in elementary torch operations, or with ``own`` the
library's entry points on the same inputs.  Layout of the 4-bit cache: one
block of 72 * d bytes per (page of 64 tokens, KV head):

    K codes   64 rows of d/2 bytes.  32-bit word (d/32) * c + j of a row
              (c < 4, j < d/32) holds columns 32 j + 8 c + i, i < 8, at bits
              16 (i % 2) + 4 (i / 2).
    V codes   32 rows of d bytes, one per pair of tokens (2u, 2u + 1).  Word
              (d/32) * r + j (r < 8) holds columns 32 j + 4 r + i, i < 4, of
              token 2u + e at bits 16 e + 4 i.
    K params  [64][d/64] words: bf16 scale (low half), bf16 minimum (high half)
    V params  likewise

and a value is scale * code + minimum of its token's group of 64 columns.
"""

import math

import torch

own = False

PAGE = 64


def listed():
    return [
        # one decode step of a full serving batch: a token each, a page boundary here and there
        dict(name="plan_step", op="plan", requests=128, cached_lo=512, cached_hi=65536, new_lo=1, new_hi=1, rows=128),
        # a step that admits many prompts beside running requests
        dict(name="plan_prompts", op="plan", requests=1024, cached_lo=0, cached_hi=8192, new_lo=1, new_hi=512,
             rows=300000),
        # a decode step's projected rows, packed by token
        dict(name="rope_step", op="rope", packed=True, batch=8, heads=16, kv_heads=8, tokens=1, dim=128, rot=128,
             interleaved=False, dtype="bf16"),
        # a prompt batch's rows before prefill
        dict(name="rope_prefill", op="rope", packed=False, batch=4, heads=16, kv_heads=16, tokens=8192, dim=128,
             rot=128, interleaved=False, dtype="bf16"),
        # gradients of a training batch
        dict(name="rope_grad", op="rope_grad", packed=False, batch=4, heads=16, kv_heads=4, tokens=8192, dim=128,
             rot=128, interleaved=False, dtype="bf16"),
        # a small fp32 model with a partial, interleaved rotation and an odd packed length
        dict(name="rope_grad_f32", op="rope_grad", packed=True, batch=1, heads=6, kv_heads=2, tokens=1001, dim=64,
             rot=32, interleaved=True, dtype="f32"),
        # the tokens of one decode step into their pages
        dict(name="append_step", op="append", sequences=128, tokens=1, kv_heads=4, dim=128),
        # two long prompts into their pages
        dict(name="append_prompts", op="append", sequences=2, tokens=8191, kv_heads=8, dim=128),
        # a few short requests of a small model
        dict(name="decode_short", op="decode", sequences=3, len_lo=1, len_hi=300, heads=6, kv_heads=2, dim=64,
             paged=True),
        # a decode step over a contiguous cache
        dict(name="decode_step", op="decode", sequences=8, len_lo=4096, len_hi=4096, heads=16, kv_heads=8, dim=128,
             paged=False),
        # a full serving batch of ragged lengths over the paged cache
        dict(name="decode_paged", op="decode", sequences=128, len_lo=512, len_hi=16384, heads=16, kv_heads=4, dim=128,
             paged=True),
        # long contexts
        dict(name="decode_long", op="decode", sequences=32, len_lo=32768, len_hi=32768, heads=32, kv_heads=8, dim=128,
             paged=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope_grad", "append", "decode", "decode"])
    if op == "plan":
        requests = _log_int(rng, 1, 1024)
        new_hi = _log_int(rng, 1, 512)
        return dict(op=op, requests=requests, cached_lo=0, cached_hi=_log_int(rng, 1, 65536), new_lo=rng.choice([0, 1]),
                    new_hi=new_hi, rows=requests * new_hi + rng.randint(0, 64))
    dim = rng.choice([64, 128])
    if op in ("rope", "rope_grad"):
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.randint(1, 4)
        packed = rng.random() < 0.5
        batch = rng.randint(1, 4)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rows = 4 * 16 * 8192 * 3 * 128 // (2 if dtype == "f32" else 1)     # elements of the largest listed case
        tokens = _log_int(rng, 1, min(8192, rows // (batch * (2 * heads + kv_heads) * dim)))
        return dict(op=op, packed=packed, batch=batch, heads=heads, kv_heads=kv_heads, tokens=tokens, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, 16]), interleaved=rng.random() < 0.3, dtype=dtype)
    if op == "append":
        kv_heads = rng.randint(1, 8)
        sequences = _log_int(rng, 1, 128)
        return dict(op=op, sequences=sequences, tokens=_log_int(rng, 1, max(1, 16382 // sequences)),
                    kv_heads=kv_heads, dim=dim)
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 4, 7, 8])
    sequences = _log_int(rng, 1, 128)
    hi = _log_int(rng, 1, min(32768, 32 * 32768 * 8 // (sequences * kv_heads)))
    return dict(op="decode", sequences=sequences, len_lo=_log_int(rng, 1, hi), len_hi=hi, heads=heads,
                kv_heads=kv_heads, dim=dim, paged=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lengths(lo, hi, n, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randint(lo, hi + 1, (n,), generator=g)


def _tables(dim, rot, positions):
    """cos and sin of position * 10000^(-2i / rot), formed in 64 bits: far positions turn many times."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


def _prepare_plan(case, seed):
    n = case["requests"]
    cached = _lengths(case["cached_lo"], case["cached_hi"], n, seed)
    new = _lengths(case["new_lo"], case["new_hi"], n, seed + 1)
    have, want = (cached + PAGE - 1) // PAGE, (cached + new + PAGE - 1) // PAGE
    width = (case["cached_hi"] + case["new_hi"]) // PAGE + 2
    pool = int(want.sum()) + 32
    g = torch.Generator()
    g.manual_seed(seed + 2)
    ids = torch.randperm(pool, generator=g).int()
    used = int(have.sum())
    table = torch.full((n, width), -1, dtype=torch.int32)
    table[torch.arange(width)[None] < have[:, None]] = ids[:used]
    return dict(cached=cached.int().cuda(), new=new.int().cuda(), table=table.cuda(), free=ids[used:].cuda(),
                rows=case["rows"], pool=pool)


def _prepare_rope(case, seed):
    g = _generator(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    B, H, K, T, d = case["batch"], case["heads"], case["kv_heads"], case["tokens"], case["dim"]

    def rows(h):
        shape = (B * T, h, d) if case["packed"] else (B, h, T, d)
        return (1.5 * torch.randn(shape, device="cuda", generator=g)).to(dt)

    def weight():
        return (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(dt)

    s = dict(q=rows(H), rho=rows(H), k=rows(K), q_weight=weight(), rho_weight=weight(), k_weight=weight(), eps=1e-6,
             interleaved=case["interleaved"])
    first = 512 if case["packed"] else 0
    span = B * T if case["packed"] else T
    s["cos"], s["sin"] = _tables(d, case["rot"], first + span)
    if case["packed"]:     # every token's own position, in no order
        s["positions"] = torch.randint(0, first + span, (B * T,), device="cuda", generator=g, dtype=torch.int32)
    else:
        s["positions"] = None
    if case["op"] == "rope_grad":
        s.update(dq=rows(H), drho=rows(H), dk=rows(K))
    return s


def _page_of_slots(sequences, tokens, seed):
    """Slots of `tokens` consecutive tokens of every sequence, its pages in a random order and its first token anywhere."""
    per = (tokens + PAGE - 1) // PAGE + 1
    g = torch.Generator()
    g.manual_seed(seed)
    pages = torch.randperm(sequences * per, generator=g).view(sequences, per)
    first = torch.randint(0, PAGE, (sequences, 1), generator=g)
    pos = first + torch.arange(tokens)[None]
    return (pages.gather(1, pos // PAGE) * PAGE + pos % PAGE).reshape(-1).cuda(), sequences * per


def _prepare_append(case, seed):
    g = _generator(seed)
    n, K, d = case["sequences"] * case["tokens"], case["kv_heads"], case["dim"]
    slots, pages = _page_of_slots(case["sequences"], case["tokens"], seed)
    # keys with an offset of their own for each channel, as attention keys have
    k = torch.randn(n, K, d, device="cuda", generator=g) + 0.5 * torch.randn(K, d, device="cuda", generator=g)
    v = torch.randn(n, K, d, device="cuda", generator=g)
    cache = torch.zeros(pages, K, 72 * d, dtype=torch.uint8, device="cuda")
    return dict(k=k.bfloat16(), v=v.bfloat16(), slots=slots, cache=cache)


def _prepare_decode(case, seed):
    g = _generator(seed)
    B, H, K, d = case["sequences"], case["heads"], case["kv_heads"], case["dim"]
    lens = _lengths(case["len_lo"], case["len_hi"], B, seed)
    longest = case["len_hi"]
    width = (longest + PAGE - 1) // PAGE
    pages = (lens + PAGE - 1) // PAGE
    pool = int(pages.sum()) if case["paged"] else B * width
    blocks = pool * K
    # Codes about normal around the middle of their range, scales and minima as
    # quantised unit-variance rows have them; independent codes are the same in any order.
    codes, groups = 64 * d, 2 * d
    cache = torch.empty(blocks, codes + 4 * groups, dtype=torch.uint8, device="cuda")
    c = torch.randn(2, blocks, codes, device="cuda", generator=g).mul_(3.2).add_(8).floor_().clamp_(0, 15)
    cache[:, :codes] = c[0].mul_(16).add_(c[1])
    scale = 0.28 * torch.exp(0.15 * torch.randn(blocks, groups, device="cuda", generator=g))
    low = -8 * scale + 0.3 * torch.randn(blocks, groups, device="cuda", generator=g)
    cache[:, codes:] = torch.stack([scale, low], -1).bfloat16().view(torch.uint8).reshape(blocks, 4 * groups)
    shape = (pool, K, 72 * d) if case["paged"] else (B, K, width, 72 * d)
    s = dict(cache=cache.view(shape), scale=1 / math.sqrt(d), longest=longest, dim=d, kv_heads=K)
    s["q"] = torch.randn(B, H, d, device="cuda", generator=g).bfloat16()
    s["rho"] = (0.3 * torch.randn(B, H, d, device="cuda", generator=g)).bfloat16()
    s["lens"] = lens.int().cuda()
    s["table"] = None
    if case["paged"]:
        gc = torch.Generator()
        gc.manual_seed(seed + 3)
        table = torch.full((B, width), -1, dtype=torch.int32)
        table[torch.arange(width)[None] < pages[:, None]] = torch.randperm(pool, generator=gc).int()
        s["table"] = table.cuda()
    return s


def prepare(case, seed):
    op = case["op"]
    if op == "plan":
        s = _prepare_plan(case, seed)
    elif op in ("rope", "rope_grad"):
        s = _prepare_rope(case, seed)
    elif op == "append":
        s = _prepare_append(case, seed)
    else:
        s = _prepare_decode(case, seed)
    s["op"] = op
    return s


# ------------------------------------------------------------------ plain forms

def _plain_plan(s):
    cached, new, table, free = s["cached"].long(), s["new"].long(), s["table"], s["free"]
    total = cached + new
    have, want = (cached + PAGE - 1) // PAGE, (total + PAGE - 1) // PAGE
    need = want - have
    end = need.cumsum(0)
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    col = torch.arange(table.shape[1], device=table.device)[None]
    fresh = (col >= have[:, None]) & (col < want[:, None])
    at = (end - need)[:, None] + col - have[:, None]
    table.copy_(torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table))
    row = torch.arange(s["rows"], device=table.device)
    req = (torch.searchsorted(cu, row, right=True) - 1).clamp(max=new.numel() - 1)
    live = row < cu[-1]
    pos = torch.where(live, cached[req] + row - cu[req], 0)
    page = table[req, pos // PAGE].long()
    slot = torch.where(live, page * PAGE + pos % PAGE, -1)
    return dict(seq_lens=total.int(), cu_seqlens=cu.int(), slots=slot, positions=torch.where(live, pos, -1).int(),
                used=end[-1:].int(), table=table)


def _angles(s, x):
    """cos and sin rows that broadcast over x's heads: [B, 1, T, rot/2] or [N, 1, rot/2]."""
    if s["positions"] is None:
        return s["cos"][:x.shape[2]], s["sin"][:x.shape[2]]
    p = s["positions"].long()
    return s["cos"][p][:, None], s["sin"][p][:, None]


def _rotate(x, cos, sin, interleaved):
    half = cos.shape[-1]
    part, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part[..., :half], part[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _plain_rope_one(s, name):
    x = s[name].float()
    cos, sin = _angles(s, x)
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s[name + "_weight"].float()
    return _rotate(n, cos, sin, s["interleaved"]).to(s[name].dtype)


def _plain_rope_grad_one(s, name):
    x, dy, w = s[name].float(), s["d" + name].float(), s[name + "_weight"].float()
    cos, sin = _angles(s, x)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
    dn = _rotate(dy, cos, -sin, s["interleaved"])
    unit = x * r
    g = dn * w
    dx = r * (g - unit * (g * unit).mean(-1, keepdim=True))
    return dx.to(s[name].dtype), (dn * unit).flatten(0, -2).sum(0)


def _plain_quantise(x):
    """Codes [N, K, d], scales and minima [N, K, d/64] of bf16 rows."""
    n, k, d = x.shape
    x = x.float().view(n, k, d // 64, 64)
    low, high = x.amin(-1), x.amax(-1)
    scale = ((high - low).double() / 15).float().bfloat16()
    # in 64 bits the quotient keeps its side of a border between two codes
    q = (x - low[..., None]).double() / scale[..., None].double()
    code = torch.where(scale[..., None] > 0, q.float().round().clamp(0, 15), 0).to(torch.uint8)
    return code.view(n, k, d), scale, low.bfloat16()


def _words(codes, bits):
    """32-bit words of codes [..., i] placed at `bits` (as int32)."""
    shift = torch.tensor(bits, device=codes.device, dtype=torch.int64)
    return (codes.long() << shift).sum(-1)


def _plain_append(s):
    cache, slots = s["cache"], s["slots"]
    P, K, _ = cache.shape
    n, _, d = s["k"].shape
    j = d // 32
    page, row = slots // PAGE, slots % PAGE
    kc, ks, kl = _plain_quantise(s["k"])
    vc, vs, vl = _plain_quantise(s["v"])
    # K: word (d/32) c + j of a row holds columns 32 j + 8 c + i
    kw = _words(kc.view(n, K, j, 4, 8).transpose(2, 3), [0, 16, 4, 20, 8, 24, 12, 28]).reshape(n, K, d // 8)
    kw = torch.where(kw >= 1 << 31, kw - (1 << 32), kw).int().contiguous().view(torch.uint8)
    # V: half e of word (d/32) r + j of a pair's row holds columns 32 j + 4 r + i
    vw = _words(vc.view(n, K, j, 8, 4).transpose(2, 3), [0, 4, 8, 12]).reshape(n, K, d // 4)
    vw = torch.where(vw >= 1 << 15, vw - (1 << 16), vw).to(torch.int16)
    kp = torch.stack([ks, kl], -1).contiguous().view(torch.uint8).view(n, K, -1)
    vp = torch.stack([vs, vl], -1).contiguous().view(torch.uint8).view(n, K, -1)
    c = d // 2 * PAGE
    g = d // 64 * 4 * PAGE
    cache[:, :, :c].view(P, K, PAGE, -1)[page, :, row] = kw
    cache[:, :, c:2 * c].view(torch.int16).view(P, K, PAGE // 2, d // 4, 2)[page, :, row // 2, :, row % 2] = vw
    cache[:, :, 2 * c:2 * c + g].view(P, K, PAGE, -1)[page, :, row] = kp
    cache[:, :, 2 * c + g:].view(P, K, PAGE, -1)[page, :, row] = vp
    # read back
    kr, vr = _plain_unpack(cache, d)
    return dict(k=kr[page, :, row], v=vr[page, :, row])


def _nibbles(words, bits):
    shift = torch.tensor(bits, device=words.device, dtype=torch.int32)
    return ((words[..., None] >> shift) & 15).to(torch.uint8)


def _plain_unpack(cache, d):
    """Blocks [..., 72 d] as the keys and values they stand for, [..., 64, d] fp32."""
    lead = cache.shape[:-1]
    j, c, g = d // 32, d // 2 * PAGE, d // 64
    kw = cache[..., :c].contiguous().view(torch.int32).view(*lead, PAGE, 4, j)
    k = _nibbles(kw, [0, 16, 4, 20, 8, 24, 12, 28]).transpose(-3, -2).reshape(*lead, PAGE, g, 64)
    vw = cache[..., c:2 * c].contiguous().view(torch.int32).view(*lead, PAGE // 2, 8, j)
    v = _nibbles(vw, [0, 4, 8, 12, 16, 20, 24, 28]).view(*lead, PAGE // 2, 8, j, 2, 4)
    v = v.movedim(-2, -4).transpose(-3, -2).reshape(*lead, PAGE, g, 64)
    p = cache[..., 2 * c:].contiguous().view(torch.bfloat16).view(*lead, 2, PAGE, g, 2).float()

    def values(code, par):
        return (code.float() * par[..., 0:1] + par[..., 1:2]).flatten(-2)

    return values(k, p[..., 0, :, :, :]), values(v, p[..., 1, :, :, :])


def _plain_decode(s):
    B, H, d = s["q"].shape
    K = s["kv_heads"]
    lens, cache = s["lens"], s["cache"]
    if s["table"] is not None:
        cache = cache[s["table"].clamp(min=0).long()].transpose(1, 2)     # [B, K, pages, 72 d]
    k, v = _plain_unpack(cache, d)
    k, v = k.flatten(2, 3), v.flatten(2, 3)
    q, rho = s["q"].float().view(B, K, -1, d), s["rho"].float().view(B, K, -1, d)
    live = (torch.arange(k.shape[2], device=k.device)[None] < lens[:, None])[:, None, None]
    score = torch.where(live, s["scale"] * (q @ k.transpose(2, 3)), -math.inf)
    probe = rho @ k.transpose(2, 3)
    e = torch.exp(score - score.amax(-1, keepdim=True))
    w = e / e.sum(-1, keepdim=True)
    mean = (w * probe).sum(-1, keepdim=True)
    return ((w * (1 + mean - probe)) @ v).view(B, H, d).bfloat16()


# ------------------------------------------------------------------ the library's calls

def _own_plan(s):
    from parallax_local_linear_b200 import binding as px
    p = px.page_plan(s["cached"], s["new"], s["table"], s["free"], num_rows=s["rows"], num_pages=s["pool"])
    return dict(seq_lens=p.seq_lens, cu_seqlens=p.cu_seqlens, slots=p.slot_map, positions=p.positions,
                used=p.pages_used, table=s["table"])


def _own_rope(s):
    from parallax_local_linear_b200 import binding as px
    return px.norm_rope(s["q"], s["rho"], s["k"], s["cos"], s["sin"], s["positions"], q_weight=s["q_weight"],
                        rho_weight=s["rho_weight"], k_weight=s["k_weight"], eps=s["eps"],
                        interleaved=s["interleaved"])


def _own_rope_grad(s):
    from parallax_local_linear_b200 import binding as px
    return px.norm_rope_backward(s["dq"], s["drho"], s["dk"], s["q"], s["rho"], s["k"], s["cos"], s["sin"],
                                 s["positions"], q_weight=s["q_weight"], rho_weight=s["rho_weight"],
                                 k_weight=s["k_weight"], eps=s["eps"], interleaved=s["interleaved"])


def _own_append(s):
    from parallax_local_linear_b200 import binding as px
    px.cache_append_q4(s["k"], s["v"], s["slots"], s["cache"])
    k, v = px.cache_gather_q4(s["cache"], s["slots"], out_dtype=torch.float32)
    return dict(k=k, v=v)


def _own_decode(s):
    from parallax_local_linear_b200 import binding as px
    return px.decode_q4(s["q"], s["rho"], s["cache"], s["scale"], seq_lens=s["lens"], page_table=s["table"],
                        kv_len=s["longest"])


def run(state):
    op = state["op"]
    if own:
        return {"plan": _own_plan, "rope": _own_rope, "rope_grad": _own_rope_grad, "append": _own_append,
                "decode": _own_decode}[op](state)
    if op == "plan":
        return _plain_plan(state)
    if op == "rope":
        return (_plain_rope_one(state, "q"), _plain_rope_one(state, "rho"), _plain_rope_one(state, "k"))
    if op == "rope_grad":
        (dq, dqw), (dr, drw), (dk, dkw) = (_plain_rope_grad_one(state, "q"), _plain_rope_grad_one(state, "rho"),
                                           _plain_rope_grad_one(state, "k"))
        return (dq, dr, dk, dqw, drw, dkw)
    if op == "append":
        return _plain_append(state)
    return _plain_decode(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "plan":
        mean_new = (case["new_lo"] + case["new_hi"]) / 2
        pages = case["requests"] * mean_new / PAGE
        return dict(bytes=16 * case["requests"] + 8 * pages + 12 * case["rows"], flops=0)
    if op in ("rope", "rope_grad"):
        size = 2 if case["dtype"] == "bf16" else 4
        rows = case["batch"] * case["tokens"] * (2 * case["heads"] + case["kv_heads"])
        turn = 4 * case["rot"] * (case["tokens"] if not case["packed"] else case["batch"] * case["tokens"])
        n = rows * case["dim"]
        if op == "rope":
            return dict(bytes=2 * n * size + turn, flops=8 * n)
        return dict(bytes=3 * n * size + turn, flops=16 * n)
    if op == "append":
        n = case["sequences"] * case["tokens"] * case["kv_heads"]
        d = case["dim"]
        # keys and values read and their codes written; the codes read and the values written
        return dict(bytes=n * (4 * d + 2 * (72 * d // 64) + 8 * d), flops=n * 2 * d * 6)
    tokens = case["sequences"] * (case["len_lo"] + case["len_hi"]) / 2
    d = case["dim"]
    return dict(bytes=tokens * case["kv_heads"] * (72 * d // 64) + 6 * case["sequences"] * case["heads"] * d,
                flops=8 * d * tokens * case["heads"])


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rope(s, grad):
    def one(name):
        x, w = s[name].double(), s[name + "_weight"].double()
        if s["positions"] is None:
            cos, sin = s["cos"].double()[:x.shape[2]], s["sin"].double()[:x.shape[2]]
        else:
            at = s["positions"].long()
            cos, sin = s["cos"].double()[at].unsqueeze(1), s["sin"].double()[at].unsqueeze(1)
        half = cos.shape[-1]
        first = torch.arange(half, device=x.device)
        a, b = (2 * first, 2 * first + 1) if s["interleaved"] else (first, first + half)
        size = torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"])
        if not grad:
            n = x / size * w
            y = n.clone()
            y[..., a] = n[..., a] * cos - n[..., b] * sin
            y[..., b] = n[..., a] * sin + n[..., b] * cos
            return y, None
        dy = s["d" + name].double()
        dn = dy.clone()
        dn[..., a] = dy[..., a] * cos + dy[..., b] * sin
        dn[..., b] = dy[..., b] * cos - dy[..., a] * sin
        # n = w x / size and d size / dx = x / (d size)
        along = (dn * w * x).sum(-1, keepdim=True)
        dx = dn * w / size - x * along / (x.shape[-1] * size ** 3)
        return dx, (dn * x / size).sum(tuple(range(x.dim() - 1)))

    (q, qw), (rho, rw), (k, kw) = one("q"), one("rho"), one("k")
    return (q, rho, k, qw, rw, kw) if grad else (q, rho, k)


def _exact_append(s):
    """Every row as its codes stand for it, apart from where they are kept."""
    def one(x):
        n, k, d = x.shape
        x = x.double().view(n, k, d // 64, 64)
        low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
        step = ((high - low) / 15).float().bfloat16().double()
        code = torch.where(step > 0, torch.round((x - low) / torch.where(step > 0, step, 1.0)), 0.0).clamp(0, 15)
        return (code * step + low).view(n, k, d)
    return dict(k=one(s["k"]), v=one(s["v"]))


def _exact_decode(s):
    B, H, d = s["q"].shape
    K, g = s["kv_heads"], H // s["kv_heads"]
    col = torch.arange(d, device="cuda")
    tok = torch.arange(PAGE, device="cuda")
    # where the code of (token, column) is: its byte in the block and its place in the byte
    kbit = 16 * (col % 2) + 4 * (col % 8 // 2)
    kword = tok[:, None] * (d // 8) + (d // 32) * (col % 32 // 8) + col // 32
    kbyte, kshift = 4 * kword + kbit // 8, (kbit % 8).expand(PAGE, d)
    vbit = 16 * (tok % 2)[:, None] + 4 * (col % 4)
    vword = (tok // 2)[:, None] * (d // 4) + (d // 32) * (col % 32 // 4) + col // 32
    vbyte, vshift = 32 * d + 4 * vword + vbit // 8, vbit % 8
    group = tok[:, None] * (d // 64) + col // 64
    lens = s["lens"].tolist()

    def unit(b, h):
        n = lens[b]
        pages = (n + PAGE - 1) // PAGE
        block = s["cache"][s["table"][b, :pages].long(), h] if s["table"] is not None else s["cache"][b, h, :pages]
        par = block[:, 64 * d:].contiguous().view(torch.bfloat16).view(pages, 2, -1, 2).double()
        k = ((block[:, kbyte] >> kshift) & 15).double() * par[:, 0, :, 0][:, group] + par[:, 0, :, 1][:, group]
        v = ((block[:, vbyte] >> vshift) & 15).double() * par[:, 1, :, 0][:, group] + par[:, 1, :, 1][:, group]
        k, v = k.reshape(-1, d)[:n], v.reshape(-1, d)[:n]
        q, rho = s["q"][b, h * g:(h + 1) * g].double(), s["rho"][b, h * g:(h + 1) * g].double()
        w = torch.softmax(s["scale"] * (q @ k.T), -1)
        kbar, vbar = w @ k, w @ v
        # vbar - (sum_i w_i (k_i - kbar)(v_i - vbar)^T)^T rho, with rho taken into the sum
        wl = w * (rho @ k.T - (rho * kbar).sum(-1, keepdim=True))
        return vbar - (wl @ v - wl.sum(-1, keepdim=True) * vbar)

    return torch.cat([unit(b, h) for b in range(B) for h in range(K)]).view(B, H, d)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None
    if case["op"] in ("rope", "rope_grad"):
        return _exact_rope(s, case["op"] == "rope_grad")
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_decode(s)
