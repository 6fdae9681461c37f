"""A prompt's way through a layer, and what is said about its tokens: more operators and what they are
measured on.

  norm    the residual's addition, the root-mean-square norm, and its output as plain numbers or as 8-bit
          integers with one scale a token (add_norm); without a norm the plain numbers of a hidden state
          to 8-bit integers (int8_quantize_rows)
  gemm    a product of such integers with 8-bit weights that have one scale a row (gemm_int8)
  append  queries and keys rotated by their tokens' positions, keys and values quantised into the paged
          microscaled cache (cache_append); in the 4-bit format the same tokens are read back, since a
          4-bit code has no tensor type of its own
  logp    log probability and rank of given tokens under rows of logits, the rows' entropy, and the
          likeliest tokens (logprobs)

The matrices, heads and vocabulary are those of the benchmark's layer and head: hidden 5120, gate and up
17408 each, 24 and 4 heads of 256 (or 48 and 8 of 128, 96 and 16 of 64), 248,320 tokens.

An 8-bit row of t has codes rint(127 t / T), in 64 bits, T its largest magnitude; after a norm t is the
sum times the weight, and the root mean square enters the scale alone.

The cache, as bytes: [pages][heads][page / 32] records of 32 tokens; a record holds K codes, V codes,
K exponents, V exponents. With p a chunk of 64 channels, a the half of the 32 tokens (token 16a + i
or 16a + 4g + t) and 32-channel block 2p + h:
  K codes      8 bit [p][a][g][i][16 channels 64p + 16g ..]     4 bit [p][g][i][a][16 channels]
  V codes      8 bit [p][a][g][i][t][4 channels 64p + 4i ..]    4 bit [p][g][i][a][t][4 channels]
  K exponents  [h][i][p][a]                                     V exponents [h][g][p][a][t]
A 4-bit byte holds the even channel in its low nibble. A block of 32 channels of one token has one
exponent byte b: its values are code * 2^(b - 127), b the smallest at which the block's largest
magnitude does not exceed the element type's largest (448 for E4M3, 6 for E2M1), at least 16. A rotated
key is rounded once to fp32 before that.
"""
import torch

own = False

MXFP8, MXFP4 = 0, 1
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


def listed():
    return [
        # four drafted tokens before the products of a decode step, which take plain numbers: latency
        dict(name="norm_step", kind="norm", rows=4, width=5120, type="f32", norm=True, residual=True, plain=True,
             codes=False),
        # a prompt before an 8-bit product
        dict(name="norm_prompt", kind="norm", rows=8192, width=5120, type="bf16", norm=True, residual=True,
             plain=False, codes=True),
        # a prompt of odd length: the hidden state before the last product
        dict(name="quantize_hidden", kind="norm", rows=4095, width=17408, type="bf16", norm=False, residual=False,
             plain=False, codes=True),
        # one token through gate and up, stacked
        dict(name="gemm_one", kind="gemm", tokens=1, rows=34816, width=5120, type="f32"),
        # the tokens of a few sequences through the last product
        dict(name="gemm_step", kind="gemm", tokens=13, rows=5120, width=17408, type="f32"),
        # a short prompt of odd length through the keys' rows
        dict(name="gemm_odd", kind="gemm", tokens=777, rows=1024, width=5120, type="f16"),
        # a long prompt through gate and up, stacked
        dict(name="gemm_prompt", kind="gemm", tokens=8192, rows=34816, width=5120, type="bf16"),
        # four drafted tokens: latency; a quarter of the channels rotates
        dict(name="append_step", kind="append", fmt=MXFP8, tokens=4, heads=4, group=6, dim=256, rot=64, page=64,
             pairs=False, type="f32"),
        # a prompt, all channels rotate
        dict(name="append_prompt", kind="append", fmt=MXFP8, tokens=16384, heads=4, group=6, dim=256, rot=256,
             page=64, pairs=False, type="bf16"),
        # a prompt of odd length into the 4-bit cache, neighbouring channels rotate together
        dict(name="append_4bit", kind="append", fmt=MXFP4, tokens=8191, heads=8, group=6, dim=128, rot=128, page=32,
             pairs=True, type="f16"),
        # one sampled token: latency
        dict(name="logp_one", kind="logp", rows=1, vocab=248320, top=20, masked=False, type="f32"),
        # a prompt's tokens scored
        dict(name="logp_prompt", kind="logp", rows=2047, vocab=248320, top=5, masked=False, type="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(lo * (hi / lo) ** rng.random() + 0.5)))


def draw(rng):
    kind = rng.choice(["norm", "gemm", "append", "logp"])
    c = dict(kind=kind, type=rng.choice(["f32", "bf16", "f16"]))
    if kind == "norm":
        norm = rng.random() < 0.7
        codes = not norm or rng.random() < 0.6
        c.update(rows=_log(rng, 1, 8192), width=_log(rng, 64, 17408), norm=norm,
                 residual=norm and rng.random() < 0.7, codes=codes, plain=norm and (not codes or rng.random() < 0.3))
        if rng.random() < 0.7:  # most widths are whole vectors
            c["width"] = max(64, c["width"] // 64 * 64)
        c["rows"] = max(1, min(c["rows"], 8192 * 5120 // c["width"]))
    elif kind == "gemm":
        c.update(tokens=_log(rng, 1, 8192), rows=_log(rng, 16, 34816), width=16 * _log(rng, 4, 1088))
        c["tokens"] = max(1, min(c["tokens"], 8192 * 34816 * 5120 // (c["rows"] * c["width"])))
    elif kind == "append":
        heads, dim = rng.choice([(4, 256), (8, 128), (16, 64), (1, 256), (2, 128), (3, 64)])
        c.update(fmt=rng.choice([MXFP8, MXFP4]), heads=heads, dim=dim, group=rng.choice([1, 2, 4, 5, 6]),
                 tokens=_log(rng, 1, 16384), page=rng.choice([32, 64, 128, 256]), pairs=rng.random() < 0.4,
                 rot=rng.choice([dim, dim, dim // 2, dim // 4, 8 * rng.randint(1, dim // 8)]))
        if c["type"] == "f32":
            c["tokens"] = min(c["tokens"], 8192)
    else:
        c.update(rows=_log(rng, 1, 2047), vocab=_log(rng, 997, 248320), top=rng.choice([0, 1, 5, 20, rng.randint(2, 64)]),
                 masked=rng.random() < 0.3)
        if c["type"] == "f32":
            c["rows"] = min(c["rows"], 1023)
    return c


# ---- the cache's bytes ----------------------------------------------------------------------------

def _record_bytes(c):
    return (66 if c["fmt"] == MXFP8 else 34) * c["dim"]


def _encode(x, fmt):
    """Codes (uint8, one a number) and exponent bytes of fp32 x[..., dim], 32 channels a block."""
    blocks = x.unflatten(-1, (-1, 32))
    bits = blocks.contiguous().view(torch.int32) & 0x7FFFFFFF
    top = bits.amax(-1)
    # the exponent field of the largest magnitude, one more where its mantissa passes the type's
    emax, most = (8, 0x600000) if fmt == MXFP8 else (2, 0x400000)
    e = ((top >> 23) - emax + ((top & 0x7FFFFF) > most).int()).clamp(min=16)
    y = torch.ldexp(blocks, (127 - e)[..., None]).flatten(-2)
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
    return torch.ldexp(v.unflatten(-1, (-1, 32)), e.int()[..., None] - 127).flatten(-2)


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


# ---- states ---------------------------------------------------------------------------------------

def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 29)
    s = dict(case=c)
    dt = TYPES[c["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if c["kind"] == "norm":
        r, n = c["rows"], c["width"]
        # a few channels stand out, and tokens differ in size
        x = normal(r, n) * (1.0 + 7.0 * (torch.rand(n, generator=gen, device=dev) > 0.99).float())
        s["x"] = (x * torch.exp(0.5 * normal(r, 1))).to(dt)
        if c["norm"]:
            s["weight"] = (1.0 + 0.2 * normal(n)).to(dt)
        if c["residual"]:
            s["residual"] = (3.0 * normal(r, n)).to(dt)
            s["sum"] = torch.empty(r, n, dtype=dt, device=dev)
        if c["plain"]:
            s["out"] = torch.empty(r, n, dtype=dt, device=dev)
        if c["codes"]:
            s["codes"] = torch.empty(r, n, dtype=torch.int8, device=dev)
            s["scales"] = torch.empty(r, device=dev)
    elif c["kind"] == "gemm":
        m, n, k = c["tokens"], c["rows"], c["width"]
        # codes of rows whose largest entry is about four times their spread
        s["a"] = torch.round(30.0 * normal(m, k)).clamp(-127, 127).to(torch.int8)
        s["w"] = torch.round(30.0 * normal(n, k)).clamp(-127, 127).to(torch.int8)
        s["a_scales"] = torch.exp(0.5 * normal(m)) / 30.0
        s["w_scales"] = torch.exp(0.3 * normal(n)) / (30.0 * k ** 0.5)
        s["out"] = torch.empty(m, n, dtype=dt, device=dev)
    elif c["kind"] == "append":
        t, h, d = c["tokens"], c["heads"], c["dim"]
        pages = -(-t // c["page"]) + 1
        order = torch.randperm(pages, generator=gen, device=dev)
        # a run of tokens that begins inside a page, over pages in mixed order
        at = torch.arange(t, device=dev) + 7 % c["page"]
        s["slots"] = order[at // c["page"]] * c["page"] + at % c["page"]
        s["positions"] = torch.arange(t, device=dev) + 1234
        angle = torch.arange(1234 + t, device=dev).double()[:, None] * torch.pow(
            torch.tensor(1e6, dtype=torch.float64, device=dev), -torch.arange(0, c["rot"], 2, device=dev) / c["rot"])
        s["rotation"] = torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()
        del angle
        s["data"] = torch.zeros(pages * h * (c["page"] // 32) * _record_bytes(c), dtype=torch.uint8, device=dev)
        s["q"] = normal(t, h * c["group"], d).to(dt)
        s["k"] = normal(t, h, d).to(dt)
        s["v"] = normal(t, h, d).to(dt)
        s["q_out"] = torch.empty_like(s["q"])
        if c["fmt"] == MXFP4:
            s["k_out"] = torch.empty(t, h, d, dtype=dt, device=dev)
            s["v_out"] = torch.empty(t, h, d, dtype=dt, device=dev)
    else:
        r, v = c["rows"], c["vocab"]
        logits = 3.0 * normal(r, v)
        if c["masked"]:  # a grammar leaves a tenth of the vocabulary
            logits = torch.where(torch.rand(v, generator=gen, device=dev) < 0.9, float("-inf"), logits)
            logits[:, v // 2] = 1.0
        s["logits"] = logits.to(dt)
        # tokens as a model gives them: near the top more often than not
        s["tokens"] = torch.argmax(logits + 2.0 * normal(r, v), -1).int()
        del logits
        s["logprob"] = torch.empty(r, device=dev)
        s["rank"] = torch.empty(r, dtype=torch.int32, device=dev)
        s["entropy"] = torch.empty(r, device=dev)
        s["top_ids"] = torch.empty(r, c["top"], dtype=torch.int32, device=dev)
        s["top_logprobs"] = torch.empty(r, c["top"], device=dev)
    return s


# ---- one pass -------------------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["kind"]](s)


def _run_own(s):
    import block_quantized_weight_pn3t_amd as pn
    c = s["case"]
    if c["kind"] == "norm":
        if c["norm"]:
            pn.add_norm(s["x"], s["weight"], EPS, out=s.get("out"), codes=s.get("codes"), scales=s.get("scales"),
                        residual=s.get("residual"), sum=s.get("sum"))
        else:
            pn.int8_quantize_rows(s["x"], s["codes"], s["scales"])
        return {name: s[name] for name in ("sum", "out", "codes", "scales") if name in s}
    if c["kind"] == "gemm":
        if "work" not in s:
            s["work"] = torch.empty(pn.gemm_int8_workspace_bytes(c["tokens"], c["rows"], c["width"]),
                                    dtype=torch.uint8, device="cuda")
        pn.gemm_int8(s["a"], s["a_scales"], s["w"], s["w_scales"], s["out"], s["work"])
        return s["out"]
    if c["kind"] == "append":
        if "cache" not in s:
            s["cache"] = pn.Cache(c["fmt"], c["heads"], c["dim"], c["page"], s["data"])
        pn.cache_append(s["cache"], s["k"], s["v"], s["slots"], s["rotation"], positions=s["positions"], q=s["q"],
                        q_out=s["q_out"], interleaved=c["pairs"])
        if c["fmt"] == MXFP8:
            return {"q": s["q_out"], **_written(s)}
        pn.cache_read(s["cache"], s["slots"], s["k_out"], s["v_out"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    if "work" not in s:
        s["work"] = torch.empty(pn.logprobs_workspace_bytes(c["rows"], c["vocab"], c["top"]), dtype=torch.uint8,
                                device="cuda")
    pn.logprobs(s["logits"], s["tokens"], s["logprob"], s["work"], rank=s["rank"], entropy=s["entropy"],
                top_ids=s["top_ids"], top_logprobs=s["top_logprobs"])
    return {name: s[name] for name in ("logprob", "rank", "entropy", "top_ids", "top_logprobs")}


def _written(s):
    """The 8-bit cache as its numbers: E4M3 codes and the exponents beside them."""
    c = s["case"]
    rec = s["data"].view(-1, _record_bytes(c))
    return {"codes": rec[:, :64 * c["dim"]].view(torch.float8_e4m3fn), "exponents": rec[:, 64 * c["dim"]:]}


def _plain_norm(s):
    c, got = s["case"], {}
    h = s["x"].float()
    if c["residual"]:
        got["sum"] = (h + s["residual"].float()).to(s["x"].dtype)
        h = got["sum"].float()
    t, r = h, 1.0
    if c["norm"]:
        r = 1.0 / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS)
        t = h * s["weight"].float()
    if c["plain"]:
        got["out"] = (t * r).to(s["x"].dtype)
    if c["codes"]:  # in 64 bits: numbers next to a border between two codes
        t = h.double() * s["weight"].double() if c["norm"] else h.double()
        top = t.abs().amax(-1, keepdim=True)
        got["codes"] = torch.round(127.0 * t / torch.where(top > 0, top, 1.0)).to(torch.int8)
        got["scales"] = (top * r / 127.0).float()[:, 0]
    return got


def _plain_gemm(s):
    acc = torch.matmul(s["a"].float(), s["w"].float().t())
    return (acc * s["a_scales"][:, None] * s["w_scales"]).to(TYPES[s["case"]["type"]])


def _turn(x, s, pairs):
    """x [tokens, heads, dim] rotated in 64 bits, rounded to fp32."""
    rot = s["rotation"].shape[1]
    row = s["rotation"][s["positions"]].double()[:, None]
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    x = x.double()
    y = x[..., :rot]
    a, b = (y[..., 0::2], y[..., 1::2]) if pairs else (y[..., :rot // 2], y[..., rot // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([y, x[..., rot:]], -1).float()


def _plain_append(s):
    c = s["case"]
    dt, h, slots, tiles = s["q"].dtype, c["heads"], s["slots"], c["page"] // 32
    q = _turn(s["q"], s, c["pairs"]).to(dt)
    parts = (*_encode(_turn(s["k"], s, c["pairs"]), c["fmt"]), *_encode(s["v"].float(), c["fmt"]))
    if c["fmt"] == MXFP4:
        return {"q": q, "k": _values(parts[0], parts[1], MXFP4).to(dt), "v": _values(parts[2], parts[3], MXFP4).to(dt)}
    # the pages hold these tokens alone: put them in their places and lay all out
    pages = s["data"].numel() // (h * tiles * _record_bytes(c))
    spread = []
    for new in parts:
        all_ = torch.zeros(pages, h, tiles * 32, new.shape[-1], dtype=torch.uint8, device=new.device)
        all_[slots // c["page"], :, slots % c["page"]] = new
        spread.append(all_.view(-1, 32, new.shape[-1]))
    s["data"].copy_(_pack(*spread, c["fmt"]).view(-1))
    return {"q": q, **_written(s)}


def _plain_logp(s):
    x = s["logits"].float()
    token = s["tokens"].long()[:, None]
    top = x.amax(-1, keepdim=True)
    d = x - top
    e = torch.exp(d)
    total = e.sum(-1)
    lse = torch.log(total)
    entropy = lse - torch.where(e > 0, e * d, 0.0).sum(-1) / total
    chosen = x.gather(1, token)
    rank = (x > chosen).sum(-1).int()
    logprob = (chosen - top)[:, 0] - lse
    del d, e
    # the order of the numbers as whole ones, the lower index first among equals
    bits = x.view(torch.int32)
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits).long() << 32
    key -= torch.arange(x.shape[1], device=x.device)
    ids = torch.topk(key, s["case"]["top"], -1)[1]
    return {"logprob": logprob, "rank": rank, "entropy": entropy, "top_ids": ids.int(),
            "top_logprobs": x.gather(1, ids) - top - lse[:, None]}


_PLAIN = {"norm": _plain_norm, "gemm": _plain_gemm, "append": _plain_append, "logp": _plain_logp}


# ---- what one pass cannot do without --------------------------------------------------------------

def work(case):
    c = case
    size = 4 if c["type"] == "f32" else 2
    if c["kind"] == "norm":
        numbers = size * (1 + 2 * c["residual"] + c["plain"]) + c["codes"]
        return {"bytes": c["rows"] * (c["width"] * numbers + 4 * c["codes"]) + c["norm"] * c["width"] * size, "flops": 0}
    if c["kind"] == "gemm":
        m, n, k = c["tokens"], c["rows"], c["width"]
        return {"bytes": (m + n) * (k + 4) + m * n * size, "flops": 2 * m * n * k}
    if c["kind"] == "append":
        token = c["heads"] * _record_bytes(c) / 32.0  # cache bytes of a token, K and V
        plain = 2 * c["heads"] * c["dim"] * size
        turned = 2 * c["heads"] * c["group"] * c["dim"] * size + 4 * c["rot"] + 16
        again = token + plain if c["fmt"] == MXFP4 else 0  # read back
        return {"bytes": c["tokens"] * (plain + token + turned + again), "flops": 0}
    return {"bytes": c["rows"] * (c["vocab"] * size + 16 + 8 * c["top"]), "flops": 0}


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
    codes), the exponent's place (in bytes), by the layout above, 8 bit."""
    t = torch.arange(32, device="cuda")[:, None]
    ch = torch.arange(c["dim"], device="cuda")[None]
    p, r, n = ch // 64, ch % 64, c["dim"] // 64
    a, h = t // 16, r // 32
    k = (((p * 2 + a) * 4 + r // 16) * 16 + t % 16) * 16 + r % 16
    v = ((((p * 2 + a) * 4 + t % 16 // 4) * 16 + r // 4) * 4 + t % 4) * 4 + r % 4 + 32 * c["dim"]
    ek = 64 * c["dim"] + ((h * 16 + t % 16) * n + p) * 2 + a
    ev = 65 * c["dim"] + (((h * 4 + t % 16 // 4) * n + p) * 2 + a) * 4 + t % 4
    return k, v, ek, ev


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
    return _EXACT[c["kind"]](c, prepare(c, seed))


def _exact_norm(c, s):
    got = {}
    h = s["x"].double()
    if c["residual"]:
        # the sum is what its type holds of it, and the norm is that of what is held
        got["sum"] = h + s["residual"].double()
        h = got["sum"].to(s["x"].dtype).double()
    y = h
    if c["norm"]:
        y = h * s["weight"].double() / (h.pow(2).sum(-1, keepdim=True) / c["width"] + EPS).sqrt()
    if c["plain"]:
        got["out"] = y
    if c["codes"]:
        got["codes"] = None
        got["scales"] = y.abs().amax(-1) / 127.0
    return got


def _exact_gemm(c, s):
    return torch.matmul(s["a"].double(), s["w"].double().t()) * (s["a_scales"].double()[:, None] * s["w_scales"].double())


def _exact_turn(x, s, pairs):
    """By one complex product a pair of channels."""
    row = s["rotation"][s["positions"]].double()
    half = row.shape[1] // 2
    turn = torch.complex(row[:, :half], row[:, half:])[:, None]
    x = x.double().clone()
    if pairs:
        z = torch.view_as_complex(x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * turn
        x[..., :2 * half] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
        x[..., :half], x[..., half:2 * half] = z.real, z.imag
    return x


def _exact_append(c, s):
    got = {"q": _exact_turn(s["q"], s, c["pairs"])}
    new = [_exact_encode(x.float(), c["fmt"]) for x in (_exact_turn(s["k"], s, c["pairs"]), s["v"])]
    if c["fmt"] == MXFP4:
        table = _numbers(c["fmt"])
        got["k"], got["v"] = (table[code] * torch.exp2((b - 127).double()).repeat_interleave(32, -1) for code, b in new)
        return got
    slots, places = s["slots"], _place(c)
    base = ((slots // c["page"])[:, None] * c["heads"] + torch.arange(c["heads"], device="cuda"))
    base = (base * (c["page"] // 32) + (slots % c["page"] // 32)[:, None]) * _record_bytes(c)
    data = s["data"].clone()
    for (code, b), code_at, exp_at in ((new[0], places[0], places[2]), (new[1], places[1], places[3])):
        data[base[..., None] + code_at[slots % 32][:, None]] = code.to(torch.uint8)
        data[base[..., None] + exp_at[slots % 32][:, None, ::32]] = b.to(torch.uint8)
    rec = data.view(-1, _record_bytes(c))
    return {**got, "codes": _numbers(MXFP8)[rec[:, :64 * c["dim"]].int()], "exponents": rec[:, 64 * c["dim"]:]}


def _exact_logp(c, s):
    """A few rows at a time, by sorting."""
    got = {"logprob": [], "entropy": [], "top_logprobs": []}
    step = max(1, (1 << 25) // c["vocab"])
    for at in range(0, c["rows"], step):
        x = s["logits"][at:at + step].double()
        x = x - torch.logsumexp(x, -1, keepdim=True)
        got["logprob"].append(x.gather(1, s["tokens"][at:at + step].long()[:, None])[:, 0])
        got["entropy"].append(-torch.special.xlogy(x.exp(), x.exp()).sum(-1))
        got["top_logprobs"].append(torch.sort(x, -1, descending=True)[0][:, :c["top"]])
    got = {name: torch.cat(parts) for name, parts in got.items()}
    return {**got, "rank": None, "top_ids": None}


_EXACT = {"norm": _exact_norm, "gemm": _exact_gemm, "append": _exact_append, "logp": _exact_logp}
