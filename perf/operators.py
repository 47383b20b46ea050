"""What the serving-step operators are measured on: building a step's page tables, returning pages,
head norm with position rotation (alone, and fused with the write into the 4-bit cache), and attention
of a chunk of tokens over the paged 4-bit cache.

``run`` computes them in plain torch operations; with ``own`` set it makes the calls of this repository's
package instead.  Both take what ``prepare`` gives.

The cache is the package's: one record of 2,304 bytes for each (page, kv head) with the 16 tokens of the
page.  K codes are 16 rows of 64 bytes, low nibble first; V codes are 8 rows of 128 bytes, row p holding
tokens 2p (low nibbles) and 2p + 1, its 16-byte group g at place (g + 2p) mod 8 with byte 2j + w for channel
16j + g + 8w; then the E4M3 scales, K as [16 tokens][8 blocks] and V as [8 rows][8 blocks][2 tokens].
"""
import math

import torch

own = False

PAGE, DIM, REC = 16, 128, 2304
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases -------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a full long-context batch: 70 requests, one new token each
        dict(name="plan_decode_b70", op="plan", batch=70, ctx_lo=24576, ctx_hi=32768, new_lo=1, new_hi=1,
             max_pages=2080, pad=0),
        # admission of prompts of very different lengths beside running requests, rows padded for a captured step
        dict(name="plan_prompts_b24", op="plan", batch=24, ctx_lo=0, ctx_hi=4093, new_lo=1, new_hi=13651,
             max_pages=10240, pad=777),
        # rejected draft tokens: a few tokens of each request go back
        dict(name="release_rejected_b70", op="release", batch=70, old_lo=24576, old_hi=32768, drop_lo=0, drop_hi=40,
             max_pages=2080),
        # long requests that end: all their pages go back
        dict(name="release_ended_b15", op="release", batch=15, old_lo=150001, old_hi=163840, drop_lo=163840,
             drop_hi=163840, max_pages=10240),
        # the queries and keys of one decode step
        dict(name="norm_rope_decode_t21", op="norm_rope", tokens=21, hq=64, hkv=8, dtype="bf16", rot=128,
             interleaved=False, norm=True, packed=True, far=8192),
        # ... and of one prefill chunk, read out of the fused projection's rows, far into a long context
        dict(name="norm_rope_chunk_t8192", op="norm_rope", tokens=8192, hq=48, hkv=8, dtype="bf16", rot=128,
             interleaved=False, norm=True, packed=True, far=163840),
        # the same fused with the write into the cache: a decode step in fp32 with a partial, interleaved rotation
        dict(name="append_decode_t70", op="append", tokens=70, each=1, hq=48, hkv=8, dtype="f32", rot=64,
             interleaved=True, norm=False, packed=False, far=32768),
        # ... and a prompt of odd length
        dict(name="append_prompt_t8191", op="append", tokens=8191, each=8191, hq=48, hkv=8, dtype="bf16", rot=128,
             interleaved=False, norm=True, packed=True, far=0),
        # attention of a few new tokens over short cached sequences: latency
        dict(name="extend_tiny_b2", op="extend", batch=2, hq=8, hkv=2, chunk_lo=3, chunk_hi=5, len_lo=255, len_hi=256,
             window=0),
        # checking 16 drafted tokens of each request at 8K context
        dict(name="extend_draft16_b12", op="extend", batch=12, hq=64, hkv=8, chunk_lo=16, chunk_hi=16, len_lo=8192,
             len_hi=8192, window=0),
        # chunks of mixed lengths in a sliding window
        dict(name="extend_window_b6", op="extend", batch=6, hq=32, hkv=8, chunk_lo=1, chunk_hi=1021, len_lo=2049,
             len_hi=12289, window=4096),
        # one prefill chunk late in a 32K context
        dict(name="extend_chunk2048_32k", op="extend", batch=1, hq=48, hkv=8, chunk_lo=2048, chunk_hi=2048,
             len_lo=32768, len_hi=32768, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "release", "norm_rope", "append", "extend", "extend"])
    if op == "plan":
        b = _log(rng, 1, 300)
        ctx = _log(rng, 1, 40000)
        new = _log(rng, 1, max(2, min(16000, 160000 // b)))
        return dict(op=op, batch=b, ctx_lo=rng.randrange(ctx + 1), ctx_hi=ctx, new_lo=rng.randrange(2), new_hi=new,
                    max_pages=(ctx + new) // PAGE + 1 + rng.randrange(100), pad=rng.randrange(200))
    if op == "release":
        b = _log(rng, 1, 300)
        old = _log(rng, 1, max(2, min(160000, 2000000 // b)))
        drop = _log(rng, 1, old + 1)
        return dict(op=op, batch=b, old_lo=rng.randrange(old + 1), old_hi=old, drop_lo=rng.randrange(drop + 1), drop_hi=drop,
                    max_pages=old // PAGE + 1 + rng.randrange(100))
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.randrange(1, 9)
    if op in ("norm_rope", "append"):
        dtype = rng.choice(["bf16", "f32"])
        most = 8192 if dtype == "bf16" else 4096
        t = _log(rng, 1, min(most, most * 48 // hq))
        c = dict(op=op, tokens=t, hq=hq, hkv=hkv, dtype=dtype, rot=rng.choice([32, 64, 96, 128]),
                 interleaved=rng.random() < 0.5, norm=rng.random() < 0.7, packed=rng.random() < 0.7,
                 far=_log(rng, 1, 1000000))
        if op == "append":
            c["each"] = rng.choice([1, _log(rng, 1, t + 1)])
        return c
    b = _log(rng, 1, 16)
    chunk = _log(rng, 1, 1500 // b)
    length = _log(rng, 16, max(17, min(32768, 98304 // b)))
    return dict(op=op, batch=b, hq=hq, hkv=hkv, chunk_lo=rng.randrange(chunk + 1), chunk_hi=chunk,
                len_lo=rng.randrange(1, length + 1), len_hi=length,
                window=rng.choice([0, 0, _log(rng, 1, length + 1)]))


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, both among them where n > 1, in a mixed order."""
    if n == 1:
        return [hi]
    step = next(s for s in (7, 11, 13, 17, 19, 23, 29) if math.gcd(s, n) == 1)
    return [lo + (hi - lo) * ((i * step) % n) // (n - 1) for i in range(n)]


def _plan_lens(c):
    return _spread(c["batch"], c["ctx_lo"], c["ctx_hi"]), _spread(c["batch"], c["new_lo"], c["new_hi"])[::-1]


def _release_lens(c):
    old = _spread(c["batch"], c["old_lo"], c["old_hi"])
    drop = _spread(c["batch"], c["drop_lo"], c["drop_hi"])[::-1]
    return old, [max(0, o - d) for o, d in zip(old, drop)]


def _extend_lens(c):
    lens = _spread(c["batch"], c["len_lo"], c["len_hi"])
    chunk = _spread(c["batch"], c["chunk_lo"], c["chunk_hi"])[::-1]
    return lens, [min(n, q) for n, q in zip(lens, chunk)]


def _append_lens(c):
    """Tokens written of each request: pieces of at most `each`."""
    t, e = c["tokens"], c["each"]
    return [e] * (t // e) + ([t % e] if t % e else [])


def _pages(n):
    return (n + PAGE - 1) // PAGE


def work(c):
    op = c["op"]
    if op == "plan":
        ctx, new = _plan_lens(c)
        t, b = sum(new), c["batch"]
        fresh = sum(_pages(x + n) - _pages(x) for x, n in zip(ctx, new))
        # lengths in; lengths, offsets, table entries, slots and positions out
        return {"bytes": 4.0 * (2 * b + 3 * b + 2 * fresh + 2 * (t + c["pad"]) + 4), "flops": 0.0}
    if op == "release":
        old, keep = _release_lens(c)
        back = sum(_pages(o) - _pages(k) for o, k in zip(old, keep))
        return {"bytes": 4.0 * (2 * c["batch"] + 2 * back + 2), "flops": 0.0}
    if op in ("norm_rope", "append"):
        t, size = c["tokens"], 2 if c["dtype"] == "bf16" else 4
        rows = t * (c["hq"] + c["hkv"])
        flops = rows * (DIM * 4.0 * c["norm"] + c["rot"] * 3.0)
        read = rows * DIM * size + 4.0 * t
        if op == "norm_rope":
            return {"bytes": read + t * DIM * (2.0 * c["hq"] + size * c["hkv"]), "flops": flops}
        read += t * c["hkv"] * DIM * size + 4.0 * t
        return {"bytes": read + t * (2.0 * DIM * c["hq"] + 144.0 * c["hkv"]), "flops": flops}
    lens, chunk = _extend_lens(c)
    pairs = keys = 0
    for n, q in zip(lens, chunk):
        for t in range(q):
            p = n - q + t
            pairs += min(p + 1, c["window"]) if c["window"] else p + 1
        first = max(0, n - q - c["window"] + 1) if c["window"] else 0
        keys += (n - first) if q else 0
    return {"bytes": keys * c["hkv"] * 144.0 + 2 * 2.0 * sum(chunk) * c["hq"] * DIM, "flops": 4.0 * DIM * pairs * c["hq"]}


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


def _quantize(x):
    """Codes (uint8, one a value) and scale bytes of rows [..., 128] in fp32: blocks of 16."""
    b = x.reshape(*x.shape[:-1], 8, 16)
    s8 = (b.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float().unsqueeze(-1)
    y = torch.where(s > 0, b / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(b))
    code = _e2m1_code(y.abs()) | (torch.signbit(y) & (s > 0)).to(torch.uint8) * 8
    return code.reshape(x.shape), s8.view(torch.uint8)


def _records(k, v):
    """Page records of K and V rows [pages, kv heads, 16, 128]."""
    n, h = k.shape[:2]
    kc, ks = _quantize(k)
    vc, vs = _quantize(v)
    kd = kc[..., 0::2] | (kc[..., 1::2] << 4)
    # [row p][group g][block j][half w] of channel 16j + g + 8w, two tokens a byte
    pair = vc.reshape(n, h, 8, 2, 8, 2, 8)                     # p, token, j, w, g
    byte = (pair[:, :, :, 0] | (pair[:, :, :, 1] << 4)).permute(0, 1, 2, 5, 3, 4).reshape(n, h, 8, 8, 16)
    vd = torch.gather(byte, 3, _places(k.device, inverse=True).view(1, 1, 8, 8, 1).expand(n, h, 8, 8, 16))
    return torch.cat([kd.reshape(n, h, 1024), vd.reshape(n, h, 1024), ks.reshape(n, h, 128),
                      vs.reshape(n, h, 8, 2, 8).transpose(3, 4).reshape(n, h, 128)], -1).contiguous()


def _places(device, inverse=False):
    """[row p][group g] -> the place of the group in its row; or [row][place] -> the group that sits there."""
    p = torch.arange(8, device=device).view(8, 1)
    g = torch.arange(8, device=device).view(1, 8)
    return (g - 2 * p) % 8 if inverse else (g + 2 * p) % 8


def _inv_freq(rot):
    return [500000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = c["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def perm(n):
        return torch.randperm(n, generator=g, device="cuda").to(torch.int32)

    s = dict(c)
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op in ("plan", "release"):
        held, _ = _plan_lens(c) if op == "plan" else _release_lens(c)
        after = [a + n for a, n in zip(*_plan_lens(c))] if op == "plan" else held
        used, need = sum(map(_pages, held)), sum(map(_pages, after))
        s["num_pages"] = need + 64
        page = perm(s["num_pages"])
        s["table"] = torch.full((c["batch"], c["max_pages"]), -1, dtype=torch.int32, device="cuda")
        count = _ints([_pages(n) for n in held])
        first = torch.cumsum(count, 0) - count
        col = torch.arange(c["max_pages"], device="cuda")
        s["table"] = torch.where(col < count[:, None], page[(first[:, None] + col).clamp(max=page.numel() - 1)], s["table"])
        s["free"] = torch.full((s["num_pages"],), -1, dtype=torch.int32, device="cuda")
        s["free"][:s["num_pages"] - used] = page[used:]
        s["num_free"] = _ints([s["num_pages"] - used])
        s["num_free_out"] = torch.empty_like(s["num_free"])
        if op == "plan":
            ctx, new = _plan_lens(c)
            s["ctx"], s["new"] = _ints(ctx), _ints(new)
            s["rows"] = sum(new) + c["pad"]
            s["seq_lens"] = torch.empty(c["batch"], dtype=torch.int32, device="cuda")
            s["q_indptr"] = torch.empty(c["batch"] + 1, dtype=torch.int32, device="cuda")
            s["kv_indptr"] = torch.empty(c["batch"], dtype=torch.int32, device="cuda")
            s["slots"] = torch.empty(s["rows"], dtype=torch.int32, device="cuda")
            s["positions"] = torch.empty(s["rows"], dtype=torch.int32, device="cuda")
        else:
            old, keep = _release_lens(c)
            s["old"], s["keep"] = _ints(old), _ints(keep)
        return s

    dt = torch.bfloat16 if c.get("dtype") != "f32" else torch.float32
    if op in ("norm_rope", "append"):
        t, hq, hkv = c["tokens"], c["hq"], c["hkv"]
        size = (normal(hq + 2 * hkv) * 0.7).exp().view(-1, 1)         # heads of different sizes
        if c["packed"]:
            # rows of the fused projection
            qkv = (normal(t, hq + 2 * hkv, DIM) * size).to(dt)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"], s["k"], s["v"] = ((normal(t, n, DIM) * size[:n]).to(dt) for n in (hq, hkv, hkv))
        s["q_weight"] = (1.0 + 0.3 * normal(DIM)).to(dt) if c["norm"] else None
        s["k_weight"] = (1.0 + 0.3 * normal(DIM)).to(dt) if c["norm"] else None
        s["inv_freq"] = _inv_freq(c["rot"])
        s["q_out"] = torch.empty((t, hq, DIM), dtype=torch.bfloat16, device="cuda")
        if op == "norm_rope":
            s["positions"] = torch.arange(t, device="cuda").to(torch.int32) + c["far"]
            s["k_out"] = torch.empty((t, hkv, DIM), dtype=dt, device="cuda")
        else:
            lens = _append_lens(c)
            # request r's tokens begin inside a page, as they do after other tokens
            start = [(5 * r + c["far"]) % PAGE for r in range(len(lens))]
            pages = [_pages(a + n) for a, n in zip(start, lens)]
            s["num_pages"] = sum(pages)
            page = perm(s["num_pages"])
            first = _indptr(pages)
            width = max(pages)
            at = torch.tensor([[min(first[r] + j, s["num_pages"] - 1) for j in range(width)] for r in range(len(lens))],
                              device="cuda")
            s["table"] = page[at].contiguous()
            r = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(lens, device="cuda"))
            inside = torch.arange(t, device="cuda") - torch.tensor(_indptr(lens)[:-1], device="cuda")[r]
            at = inside + torch.tensor(start, device="cuda")[r]
            s["slots"] = s["table"][r, at // PAGE] * PAGE + (at % PAGE).to(torch.int32)
            s["positions"] = (at + c["far"] - c["far"] % PAGE).to(torch.int32)
            s["pool"] = torch.zeros((s["num_pages"], hkv, REC), dtype=torch.uint8, device="cuda")
            s["read_lens"] = _ints([a + n for a, n in zip(start, lens)])
            rows = _indptr([a + n for a, n in zip(start, lens)])
            s["read_at"], s["read_rows"] = _ints(rows[:-1]), rows[-1]
            s["read_index"] = torch.tensor(rows[:-1], device="cuda")[r] + at
            s["k_fp8"] = torch.zeros((rows[-1], hkv, DIM), dtype=torch.uint8, device="cuda")
            s["v_fp8"] = torch.zeros_like(s["k_fp8"])
    else:
        lens, chunk = _extend_lens(c)
        width = max(map(_pages, lens)) + 1
        pages = [_pages(n) for n in lens]
        s["num_pages"] = sum(pages) + 1
        page = perm(s["num_pages"])
        first = torch.tensor(_indptr(pages)[:-1], device="cuda")
        col = torch.arange(width, device="cuda")
        s["table"] = page[(first[:, None] + col).clamp(max=s["num_pages"] - 1)].contiguous()
        hkv = c["hkv"]
        # heads of different sizes, a few channels that stand out
        k = normal(s["num_pages"], hkv, PAGE, DIM) * (0.5 + torch.rand((1, hkv, 1, 1), generator=g, device="cuda"))
        k[..., :4] *= 4.0
        v = normal(s["num_pages"], hkv, PAGE, DIM) * (0.5 + torch.rand((1, hkv, 1, 1), generator=g, device="cuda"))
        s["pool"] = _records(k, v)
        s["rows"] = sum(chunk)
        s["q"] = normal(s["rows"], c["hq"], DIM).to(torch.bfloat16)
        s["q_indptr"], s["seq_lens"] = _ints(_indptr(chunk)), _ints(lens)
        s["chunk"], s["max_len"], s["max_q_len"] = _ints(chunk), max(lens), max(chunk)
        s["out"] = torch.zeros((s["rows"], c["hq"], DIM), dtype=torch.bfloat16, device="cuda")
    if own:
        import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
        if "pool" in s:
            s["cache"] = nv.NVFP4Cache(s["pool"])
        if "inv_freq" in s:
            s["rope"] = nv.Rope(s["inv_freq"], interleaved=c["interleaved"])
        if op == "extend":
            s["workspace"] = nv.new_extend_workspace(s["rows"], s["max_q_len"], c["batch"], c["hq"], hkv,
                                                     s["table"].shape[1], window=c["window"])
    return s


# ---- the operators -----------------------------------------------------------------------------------

def run(s):
    return _own(s) if own else {"plan": _plan, "release": _release, "norm_rope": _norm_rope, "append": _append,
                                "extend": _extend}[s["op"]](s)


def _own(s):
    import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
    op = s["op"]
    if op == "plan":
        nv.nvfp4kv_plan_step(s["ctx"], s["new"], s["table"], s["num_pages"], s["free"], s["num_free"], s["num_free_out"],
                             s["seq_lens"], s["q_indptr"], s["slots"], positions=s["positions"],
                             kv_indptr=s["kv_indptr"], dev_status=s["status"])
        return dict(table=s["table"], num_free=s["num_free_out"], seq_lens=s["seq_lens"], q_indptr=s["q_indptr"],
                    kv_indptr=s["kv_indptr"], slots=s["slots"], positions=s["positions"])
    if op == "release":
        nv.nvfp4kv_release_pages(s["old"], s["keep"], s["table"], s["num_pages"], s["free"], s["num_free"],
                                 s["num_free_out"], dev_status=s["status"])
        return dict(free=s["free"], num_free=s["num_free_out"])
    if op == "norm_rope":
        nv.nvfp4kv_qk_norm_rope(s["q"], s["k"], s["positions"], s["q_out"], s["k_out"], s["rope"],
                                q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6)
        return dict(q=s["q_out"], k=s["k_out"])
    if op == "append":
        nv.nvfp4kv_qk_norm_rope_append(s["cache"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"],
                                       s["rope"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                                       dev_status=s["status"])
        # the cached rows as the extend path reads them back: in 8 bits
        nv.nvfp4kv_dequant_prefix_fp8(s["cache"], s["table"], s["read_lens"], s["read_at"], s["k_fp8"], s["v_fp8"],
                                      dev_status=s["status"])
        return dict(q=s["q_out"], k=s["k_fp8"].view(torch.float8_e4m3fn), v=s["v_fp8"].view(torch.float8_e4m3fn))
    nv.nvfp4kv_paged_extend(s["cache"], s["q"], s["q_indptr"], s["table"], s["seq_lens"], s["out"], s["workspace"],
                            max_q_len=s["max_q_len"], window=s["window"], dev_status=s["status"])
    return s["out"]


def _plan(s):
    ctx, new, table = s["ctx"].long(), s["new"].long(), s["table"]
    seq = ctx + new
    had, has = (ctx + PAGE - 1) // PAGE, (seq + PAGE - 1) // PAGE
    fresh = has - had
    before = torch.cumsum(fresh, 0) - fresh
    col = torch.arange(table.shape[1], device=table.device)
    n = (before[:, None] + col - had[:, None]).clamp(0, s["free"].numel() - 1)
    taken = s["free"][(s["num_free"].long() - 1 - n).clamp(min=0)]
    table = torch.where((col >= had[:, None]) & (col < has[:, None]), taken, table)
    end = torch.cumsum(new, 0)
    r = torch.arange(s["rows"], device=table.device)
    b = torch.searchsorted(end, r, right=True)
    live = b < ctx.numel()
    b = b.clamp(max=ctx.numel() - 1)
    pos = ctx[b] + r - (end - new)[b]
    slot = table[b, (pos // PAGE).clamp(max=table.shape[1] - 1)].long() * PAGE + pos % PAGE
    none = torch.full_like(pos, -1)
    zero = torch.zeros(1, dtype=torch.int64, device=table.device)
    return dict(table=table, num_free=(s["num_free"] - fresh.sum()).to(torch.int32), seq_lens=seq.to(torch.int32),
                q_indptr=torch.cat([zero, end]).to(torch.int32),
                kv_indptr=(torch.cumsum(ctx, 0) - ctx).to(torch.int32),
                slots=torch.where(live, slot, none).to(torch.int32),
                positions=torch.where(live, pos, none).to(torch.int32))


def _release(s):
    old, keep, table = s["old"].long(), s["keep"].long(), s["table"]
    had, has = (old + PAGE - 1) // PAGE, (keep + PAGE - 1) // PAGE
    back = had - has
    before = torch.cumsum(back, 0) - back
    col = torch.arange(table.shape[1], device=table.device)
    goes = (col >= has[:, None]) & (col < had[:, None])
    free = s["free"].clone()
    to = torch.where(goes, s["num_free"].long() + before[:, None] + col - has[:, None], free.numel())
    free = torch.cat([free, free[:1]])                        # one place more for what does not go back
    free[to.reshape(-1)] = table.reshape(-1)
    return dict(free=free[:-1], num_free=(s["num_free"] + back.sum()).to(torch.int32))


def _rotated(x, weight, s):
    """One kind of rows [tokens, heads, 128] after norm and rotation, in fp32."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    f = torch.tensor(s["inv_freq"], dtype=torch.float64, device=x.device)
    angle = s["positions"].double()[:, None, None] * f           # far positions need 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    r = 2 * f.numel()
    if s["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1)


def _norm_rope(s):
    return dict(q=_rotated(s["q"], s["q_weight"], s).to(torch.bfloat16),
                k=_rotated(s["k"], s["k_weight"], s).to(s["k"].dtype))


def _append(s):
    q = _rotated(s["q"], s["q_weight"], s).to(torch.bfloat16)
    k = _rotated(s["k"], s["k_weight"], s).to(s["k"].dtype).float()
    mags = torch.tensor(E2M1, device=k.device)

    def held(x):
        code, scale = _quantize(x)
        val = mags[(code & 7).long()] * torch.where(code > 7, -1.0, 1.0)
        val = val.unflatten(-1, (8, 16)) * scale.view(torch.float8_e4m3fn).float().unsqueeze(-1)
        out = torch.zeros((s["read_rows"],) + tuple(x.shape[1:]), device=x.device)
        out[s["read_index"]] = val.flatten(-2)
        return out.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)

    return dict(q=q, k=held(k), v=held(s["v"].float()))


def _values(rec):
    """K and V [..., 16, 128] in fp32 of page records [..., 2304]."""
    lead = rec.shape[:-1]
    mags = torch.tensor(E2M1 + tuple(-m for m in E2M1), device=rec.device)

    def scales(a):
        return a.contiguous().view(torch.float8_e4m3fn).float()

    kd = rec[..., :1024].reshape(*lead, 16, 64)
    k = torch.stack([kd & 15, kd >> 4], -1).reshape(*lead, 16, 8, 16)
    k = mags[k.long()] * scales(rec[..., 2048:2176]).reshape(*lead, 16, 8, 1)
    vd = rec[..., 1024:2048].reshape(*lead, 8, 8, 16)
    at = _places(rec.device).view(*[1] * len(lead), 8, 8, 1).expand(*lead, 8, 8, 16)
    vd = torch.gather(vd, len(lead) + 1, at).reshape(*lead, 8, 8, 8, 2)                    # p, g, j, w
    vd = vd.permute(*range(len(lead)), -4, -2, -1, -3)                                   # p, j, w, g
    v = torch.stack([vd & 15, vd >> 4], len(lead) + 1).reshape(*lead, 16, 8, 16)           # p, token, j, (w, g)
    vs = scales(rec[..., 2176:]).reshape(*lead, 8, 8, 2).transpose(-1, -2).reshape(*lead, 16, 8, 1)
    v = mags[v.long()] * vs
    return k.reshape(*lead, 16, DIM), v.reshape(*lead, 16, DIM)


def _extend(s):
    hkv, g = s["hkv"], s["hq"] // s["hkv"]
    n = _pages(s["max_len"])
    k, v = _values(s["pool"][s["table"][:, :n].long()])            # [batch, pages, kv heads, 16, 128]
    k, v = (x.transpose(1, 2).reshape(x.shape[0], hkv, n * PAGE, DIM) for x in (k, v))
    t = torch.arange(s["max_q_len"], device=k.device)
    chunk, seq, at = s["chunk"].long(), s["seq_lens"].long(), s["q_indptr"].long()
    live = t < chunk[:, None]                                      # [batch, t]
    row = torch.where(live, at[:-1, None] + t, 0)
    q = s["q"][row].float().reshape(-1, t.numel(), hkv, g, DIM).permute(0, 2, 3, 1, 4)
    score = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)) * (1.0 / math.sqrt(DIM))
    score = score.unflatten(2, (g, t.numel()))
    pos = (seq - chunk)[:, None] + t
    key = torch.arange(n * PAGE, device=k.device)
    seen = (key <= pos[..., None]) & (key < seq[:, None, None])
    if s["window"]:
        seen = seen & (key > pos[..., None] - s["window"])
    score = torch.where(seen[:, None, None], score, -float("inf"))
    top = score.amax(-1, keepdim=True)
    score = torch.exp(score - torch.where(top > -float("inf"), top, torch.zeros_like(top)))
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score.flatten(2, 3), v).unflatten(2, (g, t.numel()))
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    o = o.permute(0, 3, 1, 2, 4).reshape(-1, t.numel(), s["hq"], DIM).to(torch.bfloat16)
    out = torch.zeros((s["rows"] + 1, s["hq"], DIM), dtype=torch.bfloat16, device=o.device)
    out[torch.where(live, row, s["rows"])] = o
    return out[:-1]


# ---- the definitions in 64 bits ------------------------------------------------------------------------

def exact(c, seed):
    op = c["op"]
    if op in ("plan", "release"):
        return None
    s = prepare(c, seed)
    if op in ("norm_rope", "append"):
        def turn(x, w):
            x = x.double()
            if w is not None:
                x = w.double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / DIM + 1e-6)
            y = x.clone()
            half = c["rot"] // 2
            for i, f in enumerate(s["inv_freq"]):
                a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
                z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(x[:, :1, 0]),
                                                                      s["positions"].double()[:, None] * f)
                y[..., a], y[..., b] = z.real, z.imag
            return y
        q = turn(s["q"], s["q_weight"])
        return dict(q=q, k=turn(s["k"], s["k_weight"])) if op == "norm_rope" else dict(q=q, k=None, v=None)
    lens, chunk = _extend_lens(c)
    g = c["hq"] // c["hkv"]
    out = torch.zeros((s["rows"], c["hq"], DIM), dtype=torch.float64, device="cuda")
    mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    # byte places of every (token, channel) in a record, from the layout
    tok, ch = torch.meshgrid(torch.arange(16, device="cuda"), torch.arange(DIM, device="cuda"), indexing="ij")
    j, w, grp, p = ch // 16, (ch % 16) // 8, ch % 8, tok // 2
    places = ((tok * 64 + ch // 2, ch % 2, 2048 + tok * 8 + j),
              (1024 + p * 128 + ((grp + 2 * p) % 8) * 16 + 2 * j + w, tok % 2, 2176 + p * 16 + 2 * j + tok % 2))
    row = 0
    for b in range(c["batch"]):
        n, m = lens[b], chunk[b]
        rec = s["pool"][s["table"][b, :_pages(n)].long()]
        for h in range(c["hkv"]) if m else ():
            kv = []
            for byte, high, scale in places:
                r = rec[:, h]
                code = (r[:, byte.flatten()] >> (4 * high.flatten())) & 15
                x = mag[(code & 7).long()] * (1 - 2 * (code >> 3).double())
                sb = r[:, scale.flatten()].int()
                e, f = sb // 8, (sb % 8).double()
                x = x * torch.where(e > 0, torch.ldexp(1 + f / 8, e - 7), f / 8 * 2.0 ** -6)
                kv.append(x.reshape(-1, DIM)[:n])
            pos = torch.arange(n - m, n, device="cuda")[:, None]
            key = torch.arange(n, device="cuda")[None, :]
            hide = (key > pos) | ((key <= pos - c["window"]) if c["window"] else (key < 0))
            for i in range(g):
                q = s["q"][row:row + m, h * g + i].double()
                a = (q @ kv[0].T / math.sqrt(DIM)).masked_fill(hide, -math.inf)
                out[row:row + m, h * g + i] = torch.softmax(a, -1) @ kv[1]
        row += m
    return out
