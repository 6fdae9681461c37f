"""The operators of a decode step around its matrix products, and what they are measured on.

  write   new keys and values quantised into a paged microscaled cache (cache_write); in the 4-bit
          format the same tokens are read back, since a 4-bit code has no tensor type of its own
  read    tokens of the cache gathered back as plain numbers (cache_read)
  attend  attention of a batch's newest tokens over a prefix that all sequences share and over each
          sequence's own tokens, straight from the quantised cache (attend)
  verify  drafted tokens accepted or rejected against the target's probabilities from given random
          numbers, and the token that follows (verify)

Head layouts are those of the 6144 / 1024-row q / k / v matrices of the benchmark's layer (24 and 4
heads of 256, 48 and 8 of 128, 96 and 16 of 64); the vocabulary is the 248,320 rows of its head.

The cache, as bytes: [pages][heads][page / 32] records of 32 tokens; a record holds K codes, V codes,
K exponents, V exponents. With p a chunk of 64 channels, a the half of the 32 tokens (token 16a + i
or 16a + 4g + t) and 32-channel block 2p + h:
  K codes      8 bit [p][a][g][i][16 channels 64p + 16g ..]     4 bit [p][g][i][a][16 channels]
  V codes      8 bit [p][a][g][i][t][4 channels 64p + 4i ..]    4 bit [p][g][i][a][t][4 channels]
  K exponents  [h][i][p][a]                                     V exponents [h][g][p][a][t]
A 4-bit byte holds the even channel in its low nibble. A block of 32 channels of one token has one
exponent byte b: its values are code * 2^(b - 127), b the smallest at which the block's largest
magnitude does not exceed the element type's largest (448 for E4M3, 6 for E2M1), at least 16; a block
with a number that is not finite, or of magnitude 2^127 or more, has b = 255 and stands for NaN.
"""
import torch

own = False

MXFP8, MXFP4 = 0, 1
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the 16 tokens that the matrix products take at most, from their fp32 results
        dict(name="write_step", kind="write", fmt=MXFP8, tokens=16, heads=4, dim=256, page=64, type="f32"),
        # a prompt's keys and values
        dict(name="write_prompt", kind="write", fmt=MXFP8, tokens=16384, heads=4, dim=256, page=64, type="bf16"),
        # a prompt of odd length into the 4-bit cache, read back for what follows it in the same pass
        dict(name="write_prompt_4bit", kind="write", fmt=MXFP4, tokens=8191, heads=8, dim=128, page=32, type="f16"),
        # a few hundred tokens of a sequence taken out of the cache
        dict(name="read_window", kind="read", fmt=MXFP4, tokens=333, heads=8, dim=128, page=32, type="f32"),
        # a long sequence taken out for another layout
        dict(name="read_long", kind="read", fmt=MXFP8, tokens=32768, heads=4, dim=256, page=128, type="bf16"),
        # one token of one sequence of ordinary length: latency
        dict(name="attend_one", kind="attend", fmt=MXFP8, batch=1, drafts=1, prefix=0, own_min=1000, own_max=1000,
             heads=4, group=6, dim=256, page=64, type="f32"),
        # four drafted tokens of one sequence over a long context
        dict(name="attend_long", kind="attend", fmt=MXFP8, batch=1, drafts=4, prefix=0, own_min=130077,
             own_max=130077, heads=4, group=6, dim=256, page=64, type="f32"),
        # sixteen sequences after one system prompt, their own tokens ragged
        dict(name="attend_shared", kind="attend", fmt=MXFP8, batch=16, drafts=1, prefix=16384, own_min=1,
             own_max=777, heads=8, group=6, dim=128, page=32, type="bf16"),
        # a full batch with four drafts and the token before them, 4-bit cache, prefix of odd length
        dict(name="attend_shared_drafts", kind="attend", fmt=MXFP4, batch=32, drafts=5, prefix=32769, own_min=5,
             own_max=2000, heads=4, group=6, dim=256, page=64, type="bf16"),
        # one sequence with three drafts over the head's vocabulary
        dict(name="verify_one", kind="verify", batch=1, drafts=3, vocab=248320, type="f32", draft_probs=True),
        # a batch of them
        dict(name="verify_batch", kind="verify", batch=32, drafts=4, vocab=248320, type="f32", draft_probs=True),
        # drafts that come without probabilities (a lookup), a small odd vocabulary
        dict(name="verify_lookup", kind="verify", batch=16, drafts=7, vocab=32003, type="bf16", draft_probs=False),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(lo * (hi / lo) ** rng.random() + 0.5)))


def draw(rng):
    kind = rng.choice(["write", "read", "attend", "attend", "verify"])
    c = dict(kind=kind, type=rng.choice(["f32", "bf16", "f16"]))
    if kind == "verify":
        c.update(vocab=_log(rng, 997, 248320), batch=_log(rng, 1, 32), drafts=rng.randint(1, 8),
                 draft_probs=rng.random() < 0.7)
        c["batch"] = max(1, min(c["batch"], 160 * 248320 // (c["vocab"] * (c["drafts"] + 1))))
        return c
    heads, dim = rng.choice([(4, 256), (8, 128), (16, 64), (1, 256), (2, 128), (3, 64)])
    c.update(fmt=rng.choice([MXFP8, MXFP4]), heads=heads, dim=dim, page=rng.choice([32, 64, 128, 256]))
    if kind != "attend":
        c["tokens"] = _log(rng, 1, 16384)
        return c
    c.update(group=rng.choice([1, 2, 4, 5, 6, 8]), batch=_log(rng, 1, 32), drafts=rng.randint(1, 6),
             prefix=rng.choice([0, _log(rng, 1, 32769)]), own_min=_log(rng, 1, 64))
    c["own_max"] = _log(rng, c["own_min"], max(c["own_min"], 65536 // c["batch"]))
    return c


# ---- the cache's bytes ----------------------------------------------------------------------------

def _record_bytes(c):
    return (66 if c["fmt"] == MXFP8 else 34) * c["dim"]


def _encode(x, fmt):
    """Codes (uint8, one a number) and exponent bytes of x[..., dim], 32 channels a block."""
    x = x.float()
    blocks = x.unflatten(-1, (-1, 32))
    bits = blocks.contiguous().view(torch.int32) & 0x7FFFFFFF
    top = bits.amax(-1)
    # the exponent field of the largest magnitude, one more where its mantissa passes the type's
    emax, most = (8, 0x600000) if fmt == MXFP8 else (2, 0x400000)
    e = ((top >> 23) - emax + ((top & 0x7FFFFF) > most).int()).clamp(min=16)
    bad = (top >> 23) >= 254
    e = torch.where(bad, 255, e)
    y = torch.where(bad[..., None], 0.0, torch.ldexp(blocks, (127 - e)[..., None])).flatten(-2)
    if fmt == MXFP8:
        code = y.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        a = y.abs()
        code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
                + (a >= 3.5).int() + (a > 5.0).int() + 8 * torch.signbit(y).int()).to(torch.uint8)
    return code, e.to(torch.uint8)


def _values(code, e, fmt):
    """fp32 numbers of codes[..., dim] with exponent bytes[..., dim / 32]."""
    if fmt == MXFP8:
        v = code.view(torch.float8_e4m3fn).float()
    else:
        v = torch.tensor(E2M1 + tuple(-a for a in E2M1), device=code.device)[code.int()]
    e = e.int()[..., None]
    v = torch.ldexp(v.unflatten(-1, (-1, 32)), e - 127)
    return torch.where(e == 255, float("nan"), v).flatten(-2)


def _pack(code, e_k, code_v, e_v, fmt):
    """Records [n][bytes] of tiles[n][32 tokens][dim]: codes (one a byte) and exponents."""
    n, _, d = code.shape
    k = code.view(n, 2, 16, d // 64, 4, 16)  # n a i p g e
    v = code_v.view(n, 2, 4, 4, d // 64, 16, 4)  # n a g t p i c
    if fmt == MXFP8:
        k = k.permute(0, 3, 1, 4, 2, 5).reshape(n, -1)
        v = v.permute(0, 4, 1, 2, 5, 3, 6).reshape(n, -1)
    else:
        k = k.permute(0, 3, 4, 2, 1, 5).reshape(n, -1)
        v = v.permute(0, 4, 2, 5, 1, 3, 6).reshape(n, -1)
        k = k[:, 0::2] | (k[:, 1::2] << 4)
        v = v[:, 0::2] | (v[:, 1::2] << 4)
    ek = e_k.view(n, 2, 16, d // 64, 2).permute(0, 4, 2, 3, 1).reshape(n, -1)  # n a i p h -> h i p a
    ev = e_v.view(n, 2, 4, 4, d // 64, 2).permute(0, 5, 2, 4, 1, 3).reshape(n, -1)  # n a g t p h -> h g p a t
    return torch.cat([k, v, ek, ev], 1)


def _unpack(rec, d, fmt):
    """The inverse of _pack: K codes, K exponents, V codes, V exponents, each [n][32][...]."""
    n, c = rec.shape[0], 32 * d if fmt == MXFP8 else 16 * d
    k, v, ek, ev = rec[:, :c], rec[:, c:2 * c], rec[:, 2 * c:2 * c + d], rec[:, 2 * c + d:]
    if fmt == MXFP8:
        k = k.reshape(n, d // 64, 2, 4, 16, 16).permute(0, 2, 4, 1, 3, 5)
        v = v.reshape(n, d // 64, 2, 4, 16, 4, 4).permute(0, 2, 3, 5, 1, 4, 6)
    else:
        k = torch.stack([k & 15, k >> 4], -1).reshape(n, d // 64, 4, 16, 2, 16).permute(0, 4, 3, 1, 2, 5)
        v = torch.stack([v & 15, v >> 4], -1).reshape(n, d // 64, 4, 16, 2, 4, 4).permute(0, 4, 2, 5, 1, 3, 6)
    ek = ek.reshape(n, 2, 16, d // 64, 2).permute(0, 4, 2, 3, 1)
    ev = ev.reshape(n, 2, 4, d // 64, 2, 4).permute(0, 4, 2, 5, 3, 1)
    return tuple(t.reshape(n, 32, -1) for t in (k, ek, v, ev))


def _tokens(data, c, slots):
    """fp32 K and V [len(slots)][heads][dim] of cache slots (page * page size + place)."""
    tiles = c["page"] // 32
    data = data.view(-1, c["heads"], tiles, _record_bytes(c))
    page, place = slots // c["page"], slots % c["page"]
    page, back = torch.unique(page, return_inverse=True)
    sub = data[page]
    n = sub.shape[0]
    k, ek, v, ev = _unpack(sub.reshape(-1, sub.shape[-1]), c["dim"], c["fmt"])

    def pick(t):
        return t.view(n, c["heads"], tiles * 32, -1)[back, :, place]
    return _values(pick(k), pick(ek), c["fmt"]), _values(pick(v), pick(ev), c["fmt"])


# ---- states ---------------------------------------------------------------------------------------

def _own_lengths(c):
    """Own tokens of each sequence, spread evenly from own_min to own_max in a mixed order."""
    b = c["batch"]
    return [c["own_min"] + (c["own_max"] - c["own_min"]) * ((5 * i + 3) % b if b % 5 else i) // max(b - 1, 1)
            if b > 1 else c["own_max"] for i in range(b)]


def _filled(c, tokens, gen, dev):
    """A cache of `tokens` random tokens (whole pages), pages in order."""
    pages, h, d = -(-tokens // c["page"]), c["heads"], c["dim"]
    tiles = pages * c["page"] // 32
    # keys have channels that stand out, values do not
    out = 1.0 + 3.0 * (torch.rand(h, 1, d, generator=gen, device=dev) > 0.97).float()
    k = torch.randn(tiles, h, 32, d, generator=gen, device=dev) * out
    v = torch.randn(tiles, h, 32, d, generator=gen, device=dev)
    ck, ek = _encode(k.view(tiles * h, 32, d), c["fmt"])
    del k
    cv, ev = _encode(v.view(tiles * h, 32, d), c["fmt"])
    del v
    rec = _pack(ck, ek, cv, ev, c["fmt"])
    return rec.view(pages, c["page"] // 32, h, -1).transpose(1, 2).contiguous().view(-1)


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 17)
    s = dict(case=c)
    if c["kind"] == "verify":
        b, n, v = c["batch"], c["drafts"], c["vocab"]
        dt = TYPES[c["type"]]
        logits = 3.0 * torch.randn(b, n + 1, v, generator=gen, device=dev)
        s["p"] = torch.softmax(logits, -1).to(dt)
        q = torch.softmax(logits[:, :n] + 0.7 * torch.randn(b, n, v, generator=gen, device=dev), -1)
        del logits
        s["draft"] = torch.multinomial(q.view(b * n, v), 1, generator=gen).view(b, n).int()
        s["q"] = q.to(dt) if c["draft_probs"] else None
        if not c["draft_probs"]:  # a lookup hits the target's likeliest token more often than not
            s["draft"] = torch.where(torch.rand(b, n, generator=gen, device=dev) < 0.7,
                                     s["p"][:, :n].float().argmax(-1).int(), s["draft"])
        s["u_accept"] = torch.rand(b, n, generator=gen, device=dev)
        s["u_sample"] = torch.rand(b, generator=gen, device=dev)
        s["tokens"] = torch.empty(b, n + 1, dtype=torch.int32, device=dev)
        s["accepted"] = torch.empty(b, dtype=torch.int32, device=dev)
        return s
    h, d, dt = c["heads"], c["dim"], TYPES[c["type"]]
    if c["kind"] != "attend":
        t = c["tokens"]
        pages = -(-t // c["page"]) + 1
        order = torch.randperm(pages, generator=gen, device=dev)
        # a run of tokens that begins inside a page, over pages in mixed order
        at = torch.arange(t, device=dev) + 7 % c["page"]
        s["slots"] = order[at // c["page"]] * c["page"] + at % c["page"]
        if c["kind"] == "write":
            s["data"] = torch.zeros(pages * h * (c["page"] // 32) * _record_bytes(c), dtype=torch.uint8, device=dev)
            s["k_new"] = torch.randn(t, h, d, generator=gen, device=dev).to(dt)
            s["v_new"] = torch.randn(t, h, d, generator=gen, device=dev).to(dt)
        else:
            s["data"] = _filled(c, pages * c["page"], gen, dev)
        if c["kind"] == "read" or c["fmt"] == MXFP4:
            s["k_out"] = torch.empty(t, h, d, dtype=dt, device=dev)
            s["v_out"] = torch.empty(t, h, d, dtype=dt, device=dev)
        return s
    b, n = c["batch"], c["drafts"]
    lens = _own_lengths(c)
    prefix_pages, own_pages = -(-c["prefix"] // c["page"]), -(-max(lens) // c["page"])
    pages = prefix_pages + b * own_pages
    s["data"] = _filled(c, pages * c["page"], gen, dev)
    order = torch.randperm(pages, generator=gen, device=dev).int()
    s["prefix_table"] = order[:prefix_pages].contiguous()
    s["table"] = order[prefix_pages:].view(b, own_pages).contiguous()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    # scores of a few units, as trained heads have them
    s["query"] = (1.5 * torch.randn(b, n, h * c["group"], d, generator=gen, device=dev)).to(dt)
    s["out"] = torch.empty_like(s["query"])
    s["lse"] = torch.empty(b, n, h * c["group"], dtype=torch.float32, device=dev)
    return s


# ---- one pass -------------------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["kind"]](s)


def _run_own(s):
    import block_quantized_weight_pn3t_amd as pn
    c = s["case"]
    if c["kind"] == "verify":
        if "work" not in s:
            s["work"] = torch.empty(pn.verify_workspace_bytes(c["batch"], c["vocab"]), dtype=torch.uint8,
                                    device="cuda")
        pn.verify(s["p"], s["q"], s["draft"], s["u_accept"], s["u_sample"], s["tokens"], s["accepted"], s["work"])
        return {"tokens": s["tokens"], "accepted": s["accepted"]}
    if "cache" not in s:
        s["cache"] = pn.Cache(c["fmt"], c["heads"], c["dim"], c["page"], s["data"])
    if c["kind"] == "write":
        pn.cache_write(s["cache"], s["k_new"], s["v_new"], s["slots"])
        if c["fmt"] == MXFP8:
            return _written(s)
    if c["kind"] != "attend":
        pn.cache_read(s["cache"], s["slots"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if "work" not in s:
        s["work"] = torch.empty(pn.attend_workspace_bytes(s["cache"], s["query"], s["table"], c["prefix"]),
                                dtype=torch.uint8, device="cuda")
    pn.attend(s["cache"], s["query"], s["table"], s["lens"], s["out"], s["lse"], s["work"],
              prefix_table=s["prefix_table"], prefix_len=c["prefix"])
    return {"out": s["out"], "lse": s["lse"]}


def _written(s):
    """The 8-bit cache as its numbers: E4M3 codes and the exponents beside them."""
    c = s["case"]
    rec = s["data"].view(-1, _record_bytes(c))
    return {"codes": rec[:, :64 * c["dim"]].view(torch.float8_e4m3fn), "exponents": rec[:, 64 * c["dim"]:]}


def _plain_write(s):
    c = s["case"]
    h, d, slots = c["heads"], c["dim"], s["slots"]
    ck, ek = _encode(s["k_new"], c["fmt"])
    cv, ev = _encode(s["v_new"], c["fmt"])
    # every page of the cache is in hand: put the tokens in their places, lay all out again
    data = s["data"].view(-1, _record_bytes(c))
    parts = _unpack(data, d, c["fmt"])
    tiles = c["page"] // 32
    new = []
    for old, fresh in zip(parts, (ck, ek, cv, ev)):
        old = old.contiguous().view(-1, h, tiles * 32, old.shape[-1])
        old[slots // c["page"], :, slots % c["page"]] = fresh
        new.append(old.view(-1, 32, old.shape[-1]))
    data.copy_(_pack(*new, c["fmt"]))
    return _written(s) if c["fmt"] == MXFP8 else _plain_read(s)


def _plain_read(s):
    k, v = _tokens(s["data"], s["case"], s["slots"])
    dt = TYPES[s["case"]["type"]]
    return {"k": k.to(dt), "v": v.to(dt)}


def _plain_attend(s):
    c = s["case"]
    b, n, h, g, d = c["batch"], c["drafts"], c["heads"], c["group"], c["dim"]
    dev = s["data"].device
    most = s["table"].shape[1] * c["page"]
    at = torch.arange(most, device=dev)
    own_slots = s["table"].long()[:, at // c["page"]] * c["page"] + at % c["page"]
    ko, vo = _tokens(s["data"], c, own_slots.view(-1))
    ko = ko.view(b, most, h, d).permute(0, 2, 3, 1).reshape(b * h, d, most).contiguous()
    vo = vo.view(b, most, h, d).permute(0, 2, 1, 3).reshape(b * h, most, d).contiguous()
    q = s["query"].float() * d ** -0.5
    q = q.view(b, n, h, g, d).permute(0, 2, 1, 3, 4)  # b h n g d
    sees = at[None, None] <= (s["lens"].long()[:, None] - n + torch.arange(n, device=dev))[..., None]  # b n most
    so = torch.matmul(q.reshape(b * h, n * g, d).contiguous(), ko).view(b, h, n, g, most)
    so = torch.where(sees[:, None, :, None], so, float("-inf"))
    top = so.amax(-1)
    if c["prefix"]:
        at = torch.arange(c["prefix"], device=dev)
        kp, vp = _tokens(s["data"], c, s["prefix_table"].long()[at // c["page"]] * c["page"] + at % c["page"])
        qp = q.permute(1, 0, 2, 3, 4).reshape(h, b * n * g, d).contiguous()
        sp = torch.matmul(qp, kp.permute(1, 2, 0).contiguous()).view(h, b, n, g, -1).transpose(0, 1)
        top = torch.maximum(top, sp.amax(-1))
    top = torch.where(torch.isinf(top), 0.0, top)[..., None]
    eo = torch.exp(so - top)
    total = eo.sum(-1)
    vo = torch.where(_own_hidden(s, most)[:, None, :, None], 0.0, vo.view(b, h, most, d)).view(b * h, most, d)
    out = torch.matmul(eo.reshape(b * h, n * g, most), vo).view(b, h, n, g, d)
    if c["prefix"]:
        ep = torch.exp(sp - top)
        total = total + ep.sum(-1)
        ep = ep.transpose(0, 1).reshape(h, b * n * g, -1).contiguous()
        out = out + torch.matmul(ep, vp.transpose(0, 1).contiguous()).view(h, b, n, g, d).transpose(0, 1)
    out = torch.where(total[..., None] > 0, out / total[..., None], 0.0)
    lse = torch.log(total) + top[..., 0]
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(b, n, h * g, d).to(s["query"].dtype),
            "lse": lse.permute(0, 2, 1, 3).reshape(b, n, h * g)}


def _own_hidden(s, most):
    """Places of the own pages past a sequence's tokens: what lies there is not read."""
    return torch.arange(most, device=s["data"].device)[None] >= s["lens"].long()[:, None]


def _plain_verify(s):
    p, q, draft, u = s["p"], s["q"], s["draft"].long(), s["u_accept"].double()
    b, n = draft.shape
    px = p[:, :n].gather(2, draft[..., None])[..., 0].double()
    qx = torch.ones_like(px) if q is None else q.gather(2, draft[..., None])[..., 0].double()
    accepted = (u * qx < px).int().cumprod(1).sum(1)
    row = torch.arange(b, device=p.device)
    target = p[row, accepted].double()
    at = accepted.clamp(max=n - 1)
    if q is None:
        left = target.scatter(1, draft[row, at][:, None], 0.0)
    else:
        left = (target - q[row, at].double()).clamp(min=0.0)
    all_in = (accepted == n)[:, None]
    left = torch.where(all_in | (left.sum(1, keepdim=True) <= 0), target, left)
    total = left.cumsum(1)
    over = (total > s["u_sample"].double()[:, None] * total[:, -1:]) & (left > 0)
    places = torch.arange(p.shape[2], device=p.device)
    first = torch.where(over, places, p.shape[2]).amin(1)
    last = torch.where(left > 0, places, -1).amax(1)
    token = torch.where(first < p.shape[2], first, last)
    i = torch.arange(n + 1, device=p.device)[None]
    tokens = torch.where(i < accepted[:, None], torch.nn.functional.pad(draft, (0, 1)), -1)
    tokens = torch.where(i == accepted[:, None], token[:, None], tokens)
    return {"tokens": tokens.int(), "accepted": accepted.int()}


_PLAIN = {"write": _plain_write, "read": _plain_read, "attend": _plain_attend, "verify": _plain_verify}


# ---- what one pass cannot do without --------------------------------------------------------------

def work(case):
    c = case
    size = 4 if c["type"] == "f32" else 2
    if c["kind"] == "verify":
        # one row of the target's probabilities and one of the draft's for each sequence
        return {"bytes": c["batch"] * c["vocab"] * size * (2 if c["draft_probs"] else 1), "flops": 0}
    token = c["heads"] * _record_bytes(c) / 32.0  # cache bytes of a token, K and V
    plain = 2 * c["heads"] * c["dim"] * size
    if c["kind"] != "attend":
        both = c["kind"] == "write" and c["fmt"] == MXFP4  # written and read back
        return {"bytes": c["tokens"] * (plain + token) * (2 if both else 1), "flops": 0}
    lens = _own_lengths(c)
    rows = c["batch"] * c["drafts"] * c["heads"] * c["group"]
    sees = sum(max(0, n - c["drafts"] + 1 + i) for n in lens for i in range(c["drafts"]))
    sees = sees * c["heads"] * c["group"] + rows * c["prefix"]
    return {"bytes": (c["prefix"] + sum(lens)) * token + 2 * rows * c["dim"] * size + 4 * rows,
            "flops": 4 * sees * c["dim"]}


# ---- the definition in 64 bits --------------------------------------------------------------------

def _numbers(fmt):
    """The element type's numbers by code, from its definition."""
    if fmt == MXFP4:
        mag = [0.5 * (k & 1) if k < 2 else (1 + 0.5 * (k & 1)) * 2.0 ** ((k >> 1) - 1) for k in range(8)]
    else:
        mag = [(k & 7) * 2.0 ** -9 if k < 8 else (1 + (k & 7) / 8.0) * 2.0 ** ((k >> 3) - 7) for k in range(127)]
        mag.append(float("nan"))
    return torch.tensor(mag + [-m for m in mag], dtype=torch.float64, device="cuda")


def _place(c):
    """For token t of a record (32) and channel: the code's place in its record for K and V (in
    codes), the exponent's place (in bytes), by the layout above."""
    t = torch.arange(32, device="cuda")[:, None]
    ch = torch.arange(c["dim"], device="cuda")[None]
    p, r, n = ch // 64, ch % 64, c["dim"] // 64
    a, h = t // 16, (r // 32)
    kg, ki, ke = r // 16, t % 16, r % 16
    vg, vt, vi, vc = t % 16 // 4, t % 4, r // 4, r % 4
    if c["fmt"] == MXFP8:
        k = (((p * 2 + a) * 4 + kg) * 16 + ki) * 16 + ke
        v = ((((p * 2 + a) * 4 + vg) * 16 + vi) * 4 + vt) * 4 + vc
    else:
        k = (((p * 4 + kg) * 16 + ki) * 2 + a) * 16 + ke
        v = ((((p * 4 + vg) * 16 + vi) * 2 + a) * 4 + vt) * 4 + vc
    v = v + 32 * c["dim"]
    codes = 64 * c["dim"] if c["fmt"] == MXFP8 else 32 * c["dim"]
    ek = codes + ((h * 16 + ki) * n + p) * 2 + a
    ev = codes + c["dim"] + (((h * 4 + vg) * n + p) * 2 + a) * 4 + vt
    return k, v, ek, ev


def _exact_tokens(s, c, slots):
    """K and V of slots in 64 bits."""
    table, places = _numbers(c["fmt"]), _place(c)
    rec_bytes, tiles = _record_bytes(c), c["page"] // 32
    tok = slots % 32
    tile = slots % c["page"] // 32
    base = ((slots // c["page"])[:, None] * c["heads"] + torch.arange(c["heads"], device="cuda")) * tiles + tile[:, None]
    base = (base * rec_bytes)[..., None]
    got = []
    for code_at, exp_at in ((places[0], places[2]), (places[1], places[3])):
        at, e = code_at[tok][:, None], s["data"][base + exp_at[tok][:, None]].double()
        if c["fmt"] == MXFP8:
            code = s["data"][base + at].int()
        else:
            code = (s["data"][base + at // 2].int() >> (4 * (at % 2)).int()) & 15
        x = table[code]
        if c["fmt"] == MXFP8:
            x = torch.where((code & 127) == 127, float("nan"), x)
        got.append(torch.where(e == 255, float("nan"), x * torch.exp2(e - 127)))
    return got


def _exact_encode(x, fmt):
    """Nearest code by distance, ties to the even code, and the exponent byte, in 64 bits."""
    x = x.double().unflatten(-1, (-1, 32))
    largest, mag = (448.0, _numbers(fmt)[:127]) if fmt == MXFP8 else (6.0, _numbers(fmt)[:8])
    top = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(torch.where(top > 0, top, 1.0) / largest)
    e = torch.where(m == 0.5, e - 1, e)  # the smallest e with top <= largest * 2^e
    b = torch.where(top > 0, e + 127, 16).clamp(min=16)
    y = x.abs() * torch.exp2(127.0 - b)
    mid = (mag[1:] + mag[:-1]) / 2
    up = torch.searchsorted(mid, y.contiguous(), right=True)  # a tie counts as above its border
    tie = (up > 0) & (y == mid[(up - 1).clamp(min=0)]) & (up % 2 == 1)
    code = up - tie.long()
    code = code + torch.signbit(x).long() * (128 if fmt == MXFP8 else 8)
    return code.flatten(-2), b[..., 0]


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["kind"] == "verify":
        return _exact_verify(s)
    if c["kind"] == "read":
        k, v = _exact_tokens(s, c, s["slots"])
        return {"k": k, "v": v}
    if c["kind"] == "write":
        new = [_exact_encode(s[name], c["fmt"]) for name in ("k_new", "v_new")]
        if c["fmt"] == MXFP4:
            table = _numbers(c["fmt"])
            k, v = (table[code] * torch.exp2((b - 127).double()).repeat_interleave(32, -1) for code, b in new)
            return {"k": k, "v": v}
        slots, places = s["slots"], _place(c)
        base = ((slots // c["page"])[:, None] * c["heads"] + torch.arange(c["heads"], device="cuda"))
        base = (base * (c["page"] // 32) + (slots % c["page"] // 32)[:, None]) * _record_bytes(c)
        data = s["data"].clone()
        for (code, b), code_at, exp_at in ((new[0], places[0], places[2]), (new[1], places[1], places[3])):
            data[base[..., None] + code_at[slots % 32][:, None]] = code.to(torch.uint8)
            data[base[..., None] + exp_at[slots % 32][:, None, ::32]] = b.to(torch.uint8)
        rec = data.view(-1, _record_bytes(c))
        return {"codes": _numbers(MXFP8)[rec[:, :64 * c["dim"]].int()], "exponents": rec[:, 64 * c["dim"]:]}
    return _exact_attend(s, c)


def _exact_attend(s, c):
    b, n, h, g, d = c["batch"], c["drafts"], c["heads"], c["group"], c["dim"]
    lens = _own_lengths(c)
    query = s["query"].double().view(b, n, h, g, d)
    out = torch.zeros(b, n, h, g, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, n, h, g), float("-inf"), dtype=torch.float64, device="cuda")
    prefix = None
    if c["prefix"]:
        at = torch.arange(c["prefix"], device="cuda")
        prefix = _exact_tokens(s, c, s["prefix_table"].long()[at // c["page"]] * c["page"] + at % c["page"])
    for i in range(b):
        at = torch.arange(lens[i], device="cuda")
        k, v = _exact_tokens(s, c, s["table"][i].long()[at // c["page"]] * c["page"] + at % c["page"])
        hidden = torch.zeros(n, c["prefix"] + lens[i], dtype=torch.bool, device="cuda")
        hidden[:, c["prefix"]:] = at > lens[i] - n + torch.arange(n, device="cuda")[:, None]
        if prefix is not None:
            k, v = torch.cat([prefix[0], k]), torch.cat([prefix[1], v])
        qh = query[i].permute(1, 0, 2, 3).reshape(h, n * g, d).contiguous()
        w = torch.matmul(qh, k.permute(1, 2, 0).contiguous()) / d ** 0.5
        w = w.view(h, n, g, -1).masked_fill(hidden[None, :, None], float("-inf"))
        l = torch.logsumexp(w, -1)
        w = torch.exp(w - torch.where(torch.isinf(l), 0.0, l)[..., None]).view(h, n * g, -1)
        o = torch.matmul(w, v.transpose(0, 1).contiguous()).view(h, n, g, d)
        out[i], lse[i] = o.transpose(0, 1), l.transpose(0, 1)
    return {"out": out.view(b, n, h * g, d), "lse": lse.view(b, n, h * g)}


def _exact_verify(s):
    """Sequence by sequence, on the host."""
    b, n = s["draft"].shape
    p, draft = s["p"], s["draft"].cpu()
    u, last = s["u_accept"].double().cpu(), s["u_sample"].double().cpu()
    tokens, accepted = torch.full((b, n + 1), -1, dtype=torch.int32), torch.zeros(b, dtype=torch.int32)
    for i in range(b):
        k = 0
        while k < n:
            x = int(draft[i, k])
            qx = 1.0 if s["q"] is None else float(s["q"][i, k, x])
            if not float(u[i, k]) * qx < float(p[i, k, x]):
                break
            tokens[i, k] = x
            k += 1
        left = p[i, k].double().cpu()
        if k < n:
            rest = left.clone()
            if s["q"] is None:
                rest[int(draft[i, k])] = 0.0
            else:
                rest = torch.relu(rest - s["q"][i, k].double().cpu())
            left = rest if float(rest.sum()) > 0 else left
        run_up = torch.cumsum(left, 0)
        t = int(torch.searchsorted(run_up, last[i] * run_up[-1], right=True))
        tokens[i, k] = min(t, int(torch.nonzero(left)[-1]))
        accepted[i] = k
    return {"tokens": tokens.cuda(), "accepted": accepted.cuda()}
