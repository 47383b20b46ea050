"""What the operators around long contexts are measured on: a cache held in 8 bits with a scale for each
page and kv head (written and read back, and attention over it), and attention over the pages that a cheap
score selects for each query (the bounds of a page's keys, the selection, the attention over it).

``run`` computes them in plain torch operations; with ``own`` set it makes the calls of this repository's
package instead.  Both take what ``prepare`` gives.

Two caches, one record for each (page of 16 tokens, kv head).  The 4-bit one has 2,304 bytes: K codes in 16
rows of 64 bytes, low nibble first; V codes in 8 rows of 128 bytes, row p holding tokens 2p (low nibbles) and
2p + 1, its 16-byte group g at place (g + 2p) mod 8 with byte 2j + w for channel 16j + g + 8w; then the E4M3
scales of 16 values, K as [16 tokens][8 blocks] and V as [8 rows][8 blocks][2 tokens].  The 8-bit one has 4,128
bytes: K codes (E4M3) in 16 rows of 128 bytes, channels 16c .. 16c + 15 of token t at place (c + t) mod 8 for
even and odd t alike modulo 2; V codes in 8 rows of 256 bytes, row p holding tokens 2p and 2p + 1, the 16 bytes
of channels 8c .. 8c + 7 at place (c + f(p)) mod 16, f(p) = p mod 2 + 4 (floor(p / 2) mod 2), byte 2i + w for
channel 8c + i of token 2p + w; then the scale of K and the scale of V, powers of two, in fp32.
"""
import math

import torch

own = False

PAGE, DIM, REC4, REC8 = 16, 128, 2304, 4128
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LEAST, MOST = -100, 100                       # exponents of a page's scale


# ---- cases -------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step's new tokens into the 8-bit cache: 70 requests, one token each behind others of its
        # page, larger than those at times, and the pages read back
        dict(name="cache8_step_b70", op="cache8", batch=70, hkv=8, dtype="f32", held_lo=0, held_hi=15, new_lo=1, new_hi=1),
        # prompts of very different lengths behind a few held tokens, out of a bf16 projection, and read back as
        # a later chunk's attention wants them
        dict(name="cache8_prompts_b3", op="cache8", batch=3, hkv=8, dtype="bf16", held_lo=0, held_hi=9, new_lo=1,
             new_hi=8191),
        # attention of one new token over short sequences in 8 bits: latency
        dict(name="decode8_tiny_b2", op="decode8", batch=2, hq=8, hkv=2, q_len=1, len_lo=1, len_hi=256),
        # ... of four drafted tokens a request at 8K
        dict(name="decode8_draft4_b12", op="decode8", batch=12, hq=64, hkv=8, q_len=4, len_lo=8192, len_hi=8192),
        # ... of one token of a few long requests
        dict(name="decode8_long_b6", op="decode8", batch=6, hq=48, hkv=8, q_len=1, len_lo=131073, len_hi=163840),
        # the bounds of the pages that a decode step has written into
        dict(name="bounds_step_b70", op="bounds", cache=4, batch=70, hkv=8, len_lo=1, len_hi=1000, new_lo=1, new_hi=1),
        # ... and of whole prompts, in 4 bits and in 8
        dict(name="bounds_prompts_b15", op="bounds", cache=4, batch=15, hkv=8, len_lo=24577, len_hi=32768, new_lo=32768,
             new_hi=32768),
        dict(name="bounds8_prompt_b1", op="bounds", cache=8, batch=1, hkv=8, len_lo=163840, len_hi=163840, new_lo=163840,
             new_hi=163840),
        # one token that attends to the pages that its queries select, in a short request: latency
        dict(name="sparse_tiny_b1", op="sparse", cache=4, batch=1, hq=8, hkv=2, q_len=1, len_lo=1003, len_hi=1003,
             budget=24, first=1, last=2),
        # ... of requests of 24K to 32K tokens in 8 bits, 2,048 tokens of each looked at
        dict(name="sparse8_b12", op="sparse", cache=8, batch=12, hq=48, hkv=8, q_len=1, len_lo=24576, len_hi=32768,
             budget=128, first=1, last=4),
        # ... of three drafted tokens a request, each with pages of its own
        dict(name="sparse_draft3_b5", op="sparse", cache=4, batch=5, hq=64, hkv=8, q_len=3, len_lo=2, len_hi=16001,
             budget=96, first=1, last=2),
        # ... of long requests, 4,096 of 160K tokens looked at
        dict(name="sparse_long_b10", op="sparse", cache=4, batch=10, hq=48, hkv=8, q_len=1, len_lo=163840, len_hi=163840,
             budget=256, first=4, last=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache8", "decode8", "bounds", "sparse", "sparse"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.randrange(1, 9)
    if op == "cache8":
        b = _log(rng, 1, 200)
        new = _log(rng, 1, max(2, 8192 // b))
        held = rng.randrange(16)
        return dict(op=op, batch=b, hkv=hkv, dtype=rng.choice(["bf16", "f32"]), held_lo=rng.randrange(held + 1),
                    held_hi=held, new_lo=rng.randrange(new + 1), new_hi=new)
    if op == "bounds":
        b = _log(rng, 1, 100)
        length = _log(rng, 1, max(2, 300000 // b))
        new = _log(rng, 1, length + 1)
        return dict(op=op, cache=rng.choice([4, 8]), batch=b, hkv=hkv, len_lo=rng.randrange(length + 1), len_hi=length,
                    new_lo=rng.randrange(1, new + 1), new_hi=new)
    b = _log(rng, 1, 24)
    length = _log(rng, 1, max(2, 400000 // b))
    c = dict(op=op, batch=b, hq=hq, hkv=hkv, q_len=rng.choice([1, 1, 1, 2, 3, 5, 8]), len_lo=rng.randrange(length + 1),
             len_hi=length)
    if op == "sparse":
        budget = _log(rng, 1, min(256, 4000 // (b * c["q_len"])))
        first = rng.randrange(min(4, budget) + 1)
        c.update(cache=rng.choice([4, 8]), budget=budget, first=first, last=rng.randrange(min(8, budget - first) + 1))
    return c


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, both among them where n > 1, in a mixed order."""
    if n == 1:
        return [hi]
    step = next(s for s in (7, 11, 13, 17, 19, 23, 29) if math.gcd(s, n) == 1)
    return [lo + (hi - lo) * ((i * step) % n) // (n - 1) for i in range(n)]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _new_lens(c):
    """Held and new tokens of each request (cache8)."""
    return _spread(c["batch"], c["held_lo"], c["held_hi"]), _spread(c["batch"], c["new_lo"], c["new_hi"])[::-1]


def _bound_lens(c):
    """Lengths, and where the new tokens begin (bounds)."""
    lens, new = _spread(c["batch"], c["len_lo"], c["len_hi"]), _spread(c["batch"], c["new_lo"], c["new_hi"])[::-1]
    return lens, [max(0, n - m) for n, m in zip(lens, new)]


def work(c):
    op, b, hkv = c["op"], c["batch"], c["hkv"]
    if op == "cache8":
        held, new = _new_lens(c)
        size = 2 if c["dtype"] == "bf16" else 4
        # new rows in, codes out, codes of all rows in, rows in bf16 out
        return {"bytes": 2.0 * hkv * DIM * (sum(new) * (size + 1) + (sum(new) + sum(held)) * 3), "flops": 0.0}
    if op == "bounds":
        lens, begin = _bound_lens(c)
        pages = sum(_pages(n) - a // PAGE for n, a in zip(lens, begin) if n > a)
        tokens = sum(n - a // PAGE * PAGE for n, a in zip(lens, begin) if n > a)
        return {"bytes": hkv * (tokens * (72.0 if c["cache"] == 4 else 128.0) + pages * (2.0 * DIM + 4)), "flops": 0.0}
    lens, t, row = _spread(b, c["len_lo"], c["len_hi"]), c["q_len"], 2 * 2.0 * b * c["q_len"] * c["hq"] * DIM
    if op == "decode8":
        seen = sum(max(0, n - t + i + 1) for n in lens for i in range(t))
        return {"bytes": 256.0 * hkv * sum(lens) + row, "flops": 4.0 * DIM * c["hq"] * seen}
    pages = [_pages(n) for n in lens]
    chosen = sum(min(c["budget"], n) for n in pages)          # (of drafted tokens at least one's)
    looked = sum(min(c["budget"], _pages(max(0, n - t + i + 1))) for n in lens for i in range(t))
    rec = 144.0 if c["cache"] == 4 else 256.0
    return {"bytes": hkv * (260.0 * sum(pages) + rec * PAGE * chosen + 4.0 * c["budget"] * b * t) + row,
            "flops": 4.0 * DIM * c["hq"] * (sum(pages) * t + looked * PAGE)}


# ---- inputs ------------------------------------------------------------------------------------------

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _indptr(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _e2m1_code(a):
    """Magnitude codes of |x| <= 6, nearest, ties to the even code."""
    c = (a > 0.25).to(torch.uint8)
    for edge, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += (a >= edge) if up else (a > edge)
    return c


def _quantize4(x):
    """Codes (uint8, one a value) and scale bytes of rows [..., 128] in fp32: blocks of 16."""
    b = x.reshape(*x.shape[:-1], 8, 16)
    s8 = (b.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float().unsqueeze(-1)
    y = torch.where(s > 0, b / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(b))
    code = _e2m1_code(y.abs()) | (torch.signbit(y) & (s > 0)).to(torch.uint8) * 8
    return code.reshape(x.shape), s8.view(torch.uint8)


def _places4(device, inverse=False):
    """[row p][group g] -> the place of the group in its row; or [row][place] -> the group that sits there."""
    p = torch.arange(8, device=device).view(8, 1)
    g = torch.arange(8, device=device).view(1, 8)
    return (g - 2 * p) % 8 if inverse else (g + 2 * p) % 8


def _records4(k, v):
    """4-bit records of K and V rows [pages, kv heads, 16, 128]."""
    n, h = k.shape[:2]
    kc, ks = _quantize4(k)
    vc, vs = _quantize4(v)
    kd = kc[..., 0::2] | (kc[..., 1::2] << 4)
    pair = vc.reshape(n, h, 8, 2, 8, 2, 8)                     # p, token, j, w, g
    byte = (pair[:, :, :, 0] | (pair[:, :, :, 1] << 4)).permute(0, 1, 2, 5, 3, 4).reshape(n, h, 8, 8, 16)
    vd = torch.gather(byte, 3, _places4(k.device, inverse=True).view(1, 1, 8, 8, 1).expand(n, h, 8, 8, 16))
    return torch.cat([kd.reshape(n, h, 1024), vd.reshape(n, h, 1024), ks.reshape(n, h, 128),
                      vs.reshape(n, h, 8, 2, 8).transpose(3, 4).reshape(n, h, 128)], -1).contiguous()


def _values4(rec):
    """K and V [..., 16, 128] in fp32 of 4-bit records."""
    lead = rec.shape[:-1]
    mags = torch.tensor(E2M1 + tuple(-m for m in E2M1), device=rec.device)

    def scales(a):
        return a.contiguous().view(torch.float8_e4m3fn).float()

    kd = rec[..., :1024].reshape(*lead, 16, 64)
    k = torch.stack([kd & 15, kd >> 4], -1).reshape(*lead, 16, 8, 16)
    k = mags[k.long()] * scales(rec[..., 2048:2176]).reshape(*lead, 16, 8, 1)
    vd = rec[..., 1024:2048].reshape(*lead, 8, 8, 16)
    at = _places4(rec.device).view(*[1] * len(lead), 8, 8, 1).expand(*lead, 8, 8, 16)
    vd = torch.gather(vd, len(lead) + 1, at).reshape(*lead, 8, 8, 8, 2)                    # p, g, j, w
    vd = vd.permute(*range(len(lead)), -4, -2, -1, -3)                                   # p, j, w, g
    v = torch.stack([vd & 15, vd >> 4], len(lead) + 1).reshape(*lead, 16, 8, 16)           # p, token, j, (w, g)
    vs = scales(rec[..., 2176:]).reshape(*lead, 8, 8, 2).transpose(-1, -2).reshape(*lead, 16, 8, 1)
    v = mags[v.long()] * vs
    return k.reshape(*lead, 16, DIM), v.reshape(*lead, 16, DIM)


def _two_to(e):
    """2^e in fp32 of whole numbers e, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _over(a, top):
    """a / top in fp32, rounded once (a tensor on both sides, as a number is multiplied by a reciprocal); 0 for 0."""
    return torch.where(top > 0, torch.full_like(top, a) / top, torch.zeros_like(top))


def _scale8(top):
    """2^e, e the least whole number with top <= 448 * 2^e, within LEAST .. MOST."""
    f, x = torch.frexp(top)
    e = torch.where(f <= 0.875, x - 9, x - 8)
    e = torch.where(top > 0, e, torch.full_like(e, LEAST)).clamp(LEAST, MOST)
    return _two_to(e)


def _codes8(x, s):
    return (x / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _places8(device):
    """K: [token][chunk] -> place; V: [row][chunk] -> place."""
    t, p = torch.arange(16, device=device).view(16, 1), torch.arange(8, device=device).view(8, 1)
    f = p % 2 + 4 * ((p // 2) % 2)
    return (torch.arange(8, device=device) + t % 2) % 8, (torch.arange(16, device=device) + f) % 16


def _records8(k, v):
    """8-bit records of K and V rows [pages, kv heads, 16, 128], scales from all 16 tokens."""
    n, h = k.shape[:2]
    ks, vs = _scale8(k.abs().amax((-1, -2))), _scale8(v.abs().amax((-1, -2)))
    kc = _codes8(k, ks[..., None, None]).view(torch.uint8).reshape(n, h, 16, 8, 16)
    vc = _codes8(v, vs[..., None, None]).view(torch.uint8).reshape(n, h, 8, 2, 16, 8).permute(0, 1, 2, 4, 5, 3)
    kp, vp = (x.argsort(1) for x in _places8(k.device))
    kd = torch.gather(kc, 3, kp.view(1, 1, 16, 8, 1).expand(n, h, 16, 8, 16))
    vd = torch.gather(vc.reshape(n, h, 8, 16, 16), 3, vp.view(1, 1, 8, 16, 1).expand(n, h, 8, 16, 16))
    tail = torch.zeros((n, h, 8), device=k.device)
    tail[..., 0], tail[..., 1] = ks, vs
    return torch.cat([kd.reshape(n, h, 2048), vd.reshape(n, h, 2048), tail.view(torch.uint8)], -1).contiguous()


def _values8(rec):
    """K and V [..., 16, 128] in fp32 of 8-bit records, and their scales."""
    lead, one = rec.shape[:-1], [1] * (rec.dim() - 1)
    kp, vp = _places8(rec.device)
    kd = torch.gather(rec[..., :2048].reshape(*lead, 16, 8, 16), -2, kp.view(*one, 16, 8, 1).expand(*lead, 16, 8, 16))
    vd = torch.gather(rec[..., 2048:4096].reshape(*lead, 8, 16, 16), -2, vp.view(*one, 8, 16, 1).expand(*lead, 8, 16, 16))
    vd = vd.reshape(*lead, 8, 16, 8, 2).movedim(-1, -3).reshape(*lead, 16, DIM)
    s = rec[..., 4096:4104].contiguous().view(torch.float32)
    ks, vs = s[..., 0], s[..., 1]
    k = kd.reshape(*lead, 16, DIM).contiguous().view(torch.float8_e4m3fn).float() * ks[..., None, None]
    return k, vd.contiguous().view(torch.float8_e4m3fn).float() * vs[..., None, None], ks, vs


def _values(rec):
    return _values4(rec) if rec.shape[-1] == REC4 else _values8(rec)[:2]


def _pool(c, num_pages, normal, uniform):
    """A pool of pages: heads of different sizes, a few channels that stand out, pages that differ from one
    another as the passages of a text do."""
    hkv, make = c["hkv"], _records4 if c.get("cache") == 4 else _records8
    size = [(0.5 + uniform(1, hkv, 1, 1)) for _ in range(2)]
    pool = torch.empty((num_pages, hkv, REC4 if c.get("cache") == 4 else REC8), dtype=torch.uint8, device="cuda")
    step = max(1, 16384 // hkv)
    for p0 in range(0, num_pages, step):
        n = min(step, num_pages - p0)
        k = normal(n, hkv, PAGE, DIM) + normal(n, hkv, 1, DIM) * uniform(n, hkv, 1, 1) * 1.5
        k[..., :4] *= 4.0
        pool[p0:p0 + n] = make(k * size[0], normal(n, hkv, PAGE, DIM) * size[1])
    return pool


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, b, hkv = c["op"], c["batch"], c["hkv"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    s = dict(c)
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op == "cache8":
        held, new = _new_lens(c)
        lens = [a + n for a, n in zip(held, new)]
    elif op == "bounds":
        lens, begin = _bound_lens(c)
    else:
        lens = _spread(b, c["len_lo"], c["len_hi"])
    # each request's pages, anywhere in the pool
    pages = [_pages(n) for n in lens]
    s["num_pages"] = sum(pages) + 3
    page = torch.randperm(s["num_pages"], generator=g, device="cuda").to(torch.int32)
    first = torch.tensor(_indptr(pages)[:-1], device="cuda")
    col = torch.arange(max(pages) + 1, device="cuda")
    s["table"] = page[(first[:, None] + col).clamp(max=s["num_pages"] - 1)].contiguous()
    s["lens"], s["max_len"] = _ints(lens), max(lens)
    s["pool"] = _pool(c, s["num_pages"], normal, uniform)

    if op == "cache8":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        t = sum(new)
        # tokens of different sizes, so that a page's scale moves at times
        s["k"], s["v"] = (((normal(t, hkv, DIM)) * (0.8 * normal(t, hkv, 1)).exp()).to(dt) for _ in range(2))
        s["indptr"], s["row_at"] = _ints(_indptr(new)), _ints(_indptr(lens)[:-1])
        r = torch.repeat_interleave(torch.arange(b, device="cuda"), torch.tensor(new, device="cuda"))
        at = torch.arange(t, device="cuda") - s["indptr"][r].long() + torch.tensor(held, device="cuda")[r]
        s["held"] = torch.tensor(held, device="cuda")
        s["unit"], s["inside"] = first[r] + at // PAGE, at % PAGE        # page (numbered over the requests) and place
        s["units"] = page[:sum(pages)].long()
        s["first_unit"] = first
        q = torch.repeat_interleave(torch.arange(b, device="cuda"), torch.tensor(lens, device="cuda"))
        at = torch.arange(sum(lens), device="cuda") - s["row_at"][q].long()
        s["read_unit"], s["read_inside"] = first[q] + at // PAGE, at % PAGE
        s["k_out"] = torch.zeros((sum(lens), hkv, DIM), dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
    elif op == "bounds":
        s["begin"] = _ints(begin)
        s["bounds"] = torch.zeros((s["num_pages"], hkv, 2, DIM), dtype=torch.int8, device="cuda")
        s["steps"] = torch.zeros((s["num_pages"], hkv), device="cuda")
        touched = [(r, j) for r in range(b) if lens[r] > begin[r] for j in range(begin[r] // PAGE, pages[r])]
        r, j = (torch.tensor([t[i] for t in touched], dtype=torch.int64, device="cuda") for i in (0, 1))
        s["touched"], s["valid"] = s["table"][r, j].long(), (s["lens"].long()[r] - j * PAGE).clamp(max=PAGE)
    else:
        shape = (b, c["q_len"], c["hq"], DIM) if c["q_len"] > 1 else (b, c["hq"], DIM)
        q = normal(*shape)
        if op == "sparse":
            # queries that look for something: they lean towards some page's keys
            at = (uniform(b, hkv) * _ints(pages).clamp(min=1)[:, None]).long()
            rec = s["pool"][torch.gather(s["table"].long(), 1, at), torch.arange(hkv, device="cuda")]
            k = _values(rec)[0][:, :, 3].repeat_interleave(c["hq"] // hkv, 1)
            q = q + 0.5 * (k if c["q_len"] == 1 else k[:, None])
            s["bounds"] = torch.zeros((s["num_pages"], hkv, 2, DIM), dtype=torch.int8, device="cuda")
            s["steps"] = torch.zeros((s["num_pages"], hkv), device="cuda")
            all_valid = torch.full((s["num_pages"],), PAGE, dtype=torch.int64, device="cuda")
            ends = [(first_, n) for first_, n in zip(_indptr(pages)[:-1], lens) if n % PAGE]
            if ends:
                all_valid[page[[f + n // PAGE for f, n in ends]].long()] = torch.tensor([n % PAGE for _, n in ends],
                                                                                      device="cuda")
            for p0 in range(0, s["num_pages"], 8192):
                k = _values(s["pool"][p0:p0 + 8192])[0]
                s["bounds"][p0:p0 + 8192], s["steps"][p0:p0 + 8192] = _bounds_of(k, all_valid[p0:p0 + 8192])
            s["pages"] = torch.full((b, c["q_len"], hkv, c["budget"]), -1, dtype=torch.int32, device="cuda")
        s["q"] = q.to(torch.bfloat16)
        s["out"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    if own:
        import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
        s["kv"] = nv.NVFP4Cache(s["pool"]) if c.get("cache") == 4 else nv.FP8BlockCache(s["pool"])
        if "bounds" in s:
            s["page_bounds"] = nv.PageBounds(s["bounds"], s["steps"])
        if op in ("decode8", "sparse"):
            s["workspace"] = nv.new_workspace()
    return s


# ---- the operators -----------------------------------------------------------------------------------

def run(s):
    return _own(s) if own else {"cache8": _cache8, "decode8": _decode8, "bounds": _bounds, "sparse": _sparse}[s["op"]](s)


def _own(s):
    import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
    op = s["op"]
    if op == "cache8":
        nv.fp8bkv_append(s["kv"], s["k"], s["v"], s["indptr"], s["table"], s["lens"], dev_status=s["status"])
        nv.fp8bkv_dequant(s["kv"], s["table"], s["lens"], s["row_at"], s["k_out"], s["v_out"], dev_status=s["status"])
        return dict(k=s["k_out"], v=s["v_out"])
    if op == "decode8":
        nv.fp8bkv_paged_decode(s["kv"], s["q"], s["table"], s["lens"], s["out"], s["workspace"], dev_status=s["status"])
        return s["out"]
    if op == "bounds":
        call = nv.nvfp4kv_page_bounds if s["cache"] == 4 else nv.fp8bkv_page_bounds
        call(s["kv"], s["page_bounds"], s["table"], s["lens"], from_lens=s["begin"], dev_status=s["status"])
        return dict(bounds=s["bounds"], steps=s["steps"])
    nv.nvfp4kv_select_pages(s["page_bounds"], s["q"], s["table"], s["lens"], s["pages"], first_pages=s["first"],
                            last_pages=s["last"], dev_status=s["status"])
    call = nv.nvfp4kv_selected_decode if s["cache"] == 4 else nv.fp8bkv_selected_decode
    call(s["kv"], s["q"], s["table"], s["lens"], s["pages"], s["out"], s["workspace"], dev_status=s["status"])
    return dict(pages=s["pages"], out=s["out"])


def _cache8(s):
    """New rows into their pages, whose scale rises where they need it; the pages' rows in bf16."""
    old = _values8(s["pool"][s["units"]])                        # [pages of the requests, kv heads, 16, 128]
    holds = torch.zeros_like(s["units"])
    holds[s["first_unit"][s["held"] > 0]] = s["held"][s["held"] > 0]
    out = []
    for x, was, scale in ((s["k"], old[0], old[2]), (s["v"], old[1], old[3])):
        new = torch.zeros_like(was)
        new[s["unit"], :, s["inside"]] = x.float()
        fresh = torch.zeros((was.shape[0], PAGE), dtype=torch.bool, device=was.device)
        fresh[s["unit"], s["inside"]] = True
        need = _scale8(new.abs().amax((-1, -2)))
        scale = torch.where((holds > 0)[:, None], torch.maximum(scale, need), need)
        value = torch.where(fresh[:, None, :, None], new, was)
        value = _codes8(value, scale[..., None, None]).float() * scale[..., None, None]
        untouched = ~fresh.any(-1)                               # a request without new tokens
        value = torch.where(untouched[:, None, None, None], was, value)
        out.append(value[s["read_unit"], :, s["read_inside"]].to(torch.bfloat16))
    return dict(k=out[0], v=out[1])


def _weigh(score, v):
    """Softmax over the last axis and the sum of v; a row without keys gives zeros."""
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(top > -float("inf"), top, torch.zeros_like(top)))
    total = w.sum(-1, keepdim=True)
    return torch.matmul(w, v) / torch.where(total > 0, total, torch.ones_like(total))


def _queries(s):
    """[batch, tokens, kv heads, group, 128] in fp32, and the keys that each token sees [batch, tokens]."""
    b, t, hkv = s["batch"], s["q_len"], s["hkv"]
    q = s["q"].float().reshape(b, t, hkv, s["hq"] // hkv, DIM)
    return q, (s["lens"].long()[:, None] - t + 1 + torch.arange(t, device=q.device)).clamp(min=0)


def _decode8(s):
    q, sees = _queries(s)
    b, t, hkv, g, _ = q.shape
    n = max(1, _pages(s["max_len"]))
    k, v, _, _ = _values8(s["pool"][s["table"][:, :n].long()])     # [batch, pages, kv heads, 16, 128]
    k, v = (x.transpose(1, 2).reshape(b, hkv, n * PAGE, DIM) for x in (k, v))
    score = torch.matmul(q.transpose(1, 2).reshape(b, hkv, t * g, DIM), k.transpose(-1, -2)) * (1.0 / math.sqrt(DIM))
    score = score.unflatten(2, (t, g))
    seen = torch.arange(n * PAGE, device=k.device) < sees[..., None]
    score = torch.where(seen[:, None, :, None], score, -float("inf")).flatten(2, 3)
    o = _weigh(score, v).unflatten(2, (t, g)).transpose(1, 2)
    return o.reshape(s["q"].shape).to(torch.bfloat16)


def _bounds_of(k, valid):
    """Least and largest key of each channel over a page's tokens [pages, kv heads, 16, 128], in whole steps
    rounded outwards, and the step: 1/127 of the largest magnitude."""
    seen = (torch.arange(PAGE, device=k.device) < valid[:, None])[:, None, :, None]
    hi = torch.where(seen, k, -float("inf")).amax(2)
    lo = torch.where(seen, k, float("inf")).amin(2)
    top = torch.maximum(hi.abs(), lo.abs()).amax(-1)
    r = _over(127.0, top)[..., None]
    ints = torch.stack([(lo * r).floor().clamp(min=-127.0), (hi * r).ceil().clamp(max=127.0)], 2)
    return ints.to(torch.int8), top / torch.full_like(top, 127.0)


def _bounds(s):
    out = dict(bounds=s["bounds"].clone(), steps=s["steps"].clone())
    out["bounds"][s["touched"]], out["steps"][s["touched"]] = _bounds_of(_values(s["pool"][s["touched"]])[0], s["valid"])
    return out


def _sparse(s):
    q, sees = _queries(s)
    b, t, hkv, g, _ = q.shape
    n, budget = max(1, _pages(s["max_len"])), s["budget"]
    table = s["table"][:, :n].long()
    # scores: queries in whole steps against the bounds, exact in fp32
    top = q.abs().amax((-1, -2), keepdim=True)
    w = torch.round(q * _over(127.0, top)).clamp(-127.0, 127.0)
    w = w.transpose(1, 2).reshape(b, hkv, t * g, DIM)
    ints = s["bounds"][table].permute(0, 2, 3, 4, 1).float()                          # b, hkv, 2, 128, pages
    score = torch.matmul(w.clamp(max=0.0), ints[:, :, 0]) + torch.matmul(w.clamp(min=0.0), ints[:, :, 1])
    score = score.unflatten(2, (t, g)).amax(3) * s["steps"][table].transpose(1, 2)[:, :, None]
    # first and last pages, then by score, ties to the lower page
    page = torch.arange(n, device=q.device)
    there = ((sees + PAGE - 1) // PAGE)[:, None, :, None]                                # b, 1, t, 1
    score = torch.where((page < s["first"]) | (page >= there - s["last"]), float("inf"), score)
    score = torch.where(page < there, score, -float("inf"))
    order = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :budget]
    order = torch.where(order < there, order, n)
    order = torch.cat([order, torch.full((b, hkv, t, max(0, budget - n)), n, device=q.device)], -1)
    order = torch.sort(order, dim=-1)[0].transpose(1, 2)                                 # b, t, hkv, budget
    pages = torch.where(order < n, order, -1)
    # attention over them
    at = torch.gather(table[:, None, None].expand(b, t, hkv, n), 3, pages.clamp(min=0))
    k, v = _values(s["pool"][at, torch.arange(hkv, device=q.device)[:, None]])
    k, v = k.flatten(3, 4), v.flatten(3, 4)
    key = (pages[..., None] * PAGE + torch.arange(PAGE, device=q.device)).flatten(-2)
    seen = (key >= 0) & (key < sees[:, :, None, None]) & (pages >= 0).repeat_interleave(PAGE, -1)
    score = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(DIM))
    o = _weigh(torch.where(seen[:, :, :, None], score, -float("inf")), v)
    return dict(pages=pages.to(torch.int32), out=o.reshape(s["q"].shape).to(torch.bfloat16))


# ---- the definitions in 64 bits ------------------------------------------------------------------------

def _pow2(e):
    """2^e in 64 bits of whole numbers e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(byte):
    """Values in 64 bits of E4M3 bytes."""
    x = byte.int()
    e, f = (x >> 3) & 15, (x & 7).double()
    m = torch.where(e > 0, (1 + f / 8) * _pow2(e - 7), f / 512)
    return m * (1 - 2 * (x >> 7).double())


def _cached(s, table, h):
    """K and V [tokens, 128] in 64 bits of kv head h in the pages of a table, from the layouts."""
    tok, ch = torch.meshgrid(torch.arange(16, device="cuda"), torch.arange(DIM, device="cuda"), indexing="ij")
    r, p, w = s["pool"][table.long(), h], tok // 2, tok % 2
    if r.shape[-1] == REC8:
        f = p % 2 + 4 * ((p // 2) % 2)
        places = (tok * 128 + (ch // 16 + w) % 8 * 16 + ch % 16, 2048 + p * 256 + (ch // 8 + f) % 16 * 16 + ch % 8 * 2 + w)
        s2 = r[:, 4096:4104].contiguous().view(torch.float32).double()
        return [(_e4m3(r[:, at.flatten()]) * s2[:, i:i + 1]).reshape(-1, DIM) for i, at in enumerate(places)]
    mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    j, half, grp = ch // 16, (ch % 16) // 8, ch % 8
    out = []
    for byte, high, scale in ((tok * 64 + ch // 2, ch % 2, 2048 + tok * 8 + j),
                              (1024 + p * 128 + ((grp + 2 * p) % 8) * 16 + 2 * j + half, w, 2176 + p * 16 + 2 * j + w)):
        code = (r[:, byte.flatten()] >> (4 * high.flatten())) & 15
        out.append((mag[(code & 7).long()] * (1 - 2 * (code >> 3).double()) * _e4m3(r[:, scale.flatten()])).reshape(-1, DIM))
    return out


def _attend(q, k, v):
    a = q.double() @ k.T / math.sqrt(DIM)
    return torch.softmax(a, -1) @ v


def exact(c, seed):
    s, op = prepare(c, seed), c["op"]
    if op == "cache8":
        held, new = _new_lens(c)
        out = {}
        for i, name in enumerate(("k", "v")):
            rows, r = [], 0
            for b in range(c["batch"]):
                n, m = held[b], new[b]
                for h in range(c["hkv"]):
                    x = _cached(s, s["table"][b, :max(1, _pages(n))], h)[i][:n]
                    x = torch.cat([x, s[name][r:r + m, h].double()])
                    if m == 0:
                        rows.append((b, h, x))
                        continue
                    x = torch.nn.functional.pad(x, (0, 0, 0, -x.shape[0] % PAGE)).reshape(-1, PAGE, DIM)
                    added = x.clone()
                    added[0, :n] = 0
                    top = added.abs().amax((1, 2))
                    e = torch.ceil(torch.log2((top / 448).clamp(min=1e-30)))
                    # (the logarithm may be one off)
                    e = e - (top <= 448 * _pow2(e - 1)).double() + (top > 448 * _pow2(e)).double()
                    e = e.clamp(LEAST, MOST)
                    if n:
                        old = s["pool"][s["table"][b, 0].long(), h, 4096 + 4 * i:4100 + 4 * i].view(torch.float32)
                        e[0] = torch.maximum(e[0], torch.frexp(old.double())[1][0] - 1)
                    y = x / _pow2(e)[:, None, None]
                    place = _pow2(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)     # the last place of E4M3
                    y = torch.round(y / place) * place * _pow2(e)[:, None, None]
                    rows.append((b, h, y.reshape(-1, DIM)[:n + m]))
                r += m
            at = _indptr([a + n for a, n in zip(held, new)])
            full = torch.zeros((at[-1], c["hkv"], DIM), dtype=torch.float64, device="cuda")
            for b, h, x in rows:
                full[at[b]:at[b + 1], h] = x
            out[name] = full
        return out
    if op == "bounds":
        steps = torch.zeros((s["num_pages"], c["hkv"]), dtype=torch.float64, device="cuda")
        lens, begin = _bound_lens(c)
        for b in range(c["batch"]):
            for h in range(c["hkv"]) if lens[b] > begin[b] else ():
                j = begin[b] // PAGE
                k = _cached(s, s["table"][b, j:_pages(lens[b])], h)[0].clone()
                k[lens[b] - j * PAGE:] = 0
                steps[s["table"][b, j:_pages(lens[b])].long(), h] = k.abs().reshape(-1, PAGE * DIM).amax(1) / 127
        return dict(bounds=None, steps=steps)
    lens, t, g = _spread(c["batch"], c["len_lo"], c["len_hi"]), c["q_len"], c["hq"] // c["hkv"]
    q = s["q"].reshape(c["batch"], t, c["hq"], DIM)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        table = s["table"][b, :_pages(lens[b])]
        for h in range(c["hkv"]) if lens[b] else ():
            if op == "decode8":
                k, v = _cached(s, table, h)
            for i in range(t):
                n = lens[b] - t + i + 1
                if n <= 0:
                    continue
                mine = q[b, i, h * g:(h + 1) * g]
                if op == "decode8":
                    out[b, i, h * g:(h + 1) * g] = _attend(mine, k[:n], v[:n])
                    continue
                # the selection as it is defined: whole numbers, one product in 32 bits
                num = _pages(n)
                low, high = (s["bounds"][table[:num].long(), h, x].double() for x in (0, 1))
                x = mine.float()
                x = torch.round(x * _over(127.0, x.abs().max())).double()
                best = torch.stack([torch.maximum(y * low, y * high).sum(-1) for y in x]).amax(0)
                best = (best.float() * s["steps"][table[:num].long(), h]).cpu().numpy()
                best[:c["first"]] = math.inf
                best[max(0, num - c["last"]):] = math.inf
                picked = sorted(sorted(range(num), key=lambda z: (-best[z], z))[:c["budget"]])
                k, v = _cached(s, table[picked], h)
                key = (torch.tensor(picked, device="cuda")[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()
                out[b, i, h * g:(h + 1) * g] = _attend(mine, k[key < n], v[key < n])
    out = out.reshape(s["q"].shape)
    return out if op == "decode8" else dict(pages=None, out=out)
