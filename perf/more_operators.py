"""Cases of the paged 8-bit KV cache's operators, in plain torch and through libhybrid.so.

The plain forms compute each operator from its definition with elementary
tensor operations; with ``own`` set, ``run`` makes the calls of
include/hybrid.h that a user's program makes.

The cache: 16 consecutive positions of one kv head are a block.  Rows (k after
the rotation, v as projected) are rounded to bf16.  A block whose 16 rows are
there is closed: int8 codes c and one FP32 scale s for its K and for its V,
value s * c, with a = max |x| over the block, s = a / 127 and c =
round-half-even(x * (127 / a)) clamped to [-127, 127] (these few FP32
operations are the format's definition).  The rows of a sequence's last, open
block stay bf16 in its tail until the block closes.  Pages of page_tokens
positions hold the closed blocks of all kv heads; a table gives each
sequence's pages.

A query at position t sees the positions u <= t with u < sinks or u > t -
window (window 0: every u <= t).
"""
import math
import random

import torch

own = False

APPEND, DECODE, PROMPT = "kv_append_p8", "attention_p8", "attention_p8_prompt"
BLOCK = 16


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a single row appended outside the attention call (a sequence being forced along): launch latency
        dict(name="append one row", op=APPEND, batch=1, t_lo=4096, t_hi=4096, n_lo=1, n_hi=1, nq=16, nkv=4, hd=128, page=128),
        # chunks of eight prompts of unlike lengths, MoE 35B-A3B-shaped attention layer
        dict(name="append moe b8 ragged", op=APPEND, batch=8, t_lo=0, t_hi=16384, n_lo=1, n_hi=511, nq=16, nkv=2, hd=256, page=128),
        # four full prompt chunks of the dense 4B-shaped model
        dict(name="append dense-4b 4x2048", op=APPEND, batch=4, t_lo=2048, t_hi=32768, n_lo=2048, n_hi=2048, nq=16, nkv=4, hd=128,
             page=128),
        # one token of the tiny two-layer hybrid early in its context: latency
        dict(name="decode tiny", op=DECODE, batch=1, t_lo=37, t_hi=37, window=0, sinks=0, nq=4, nkv=2, hd=64, page=128),
        # the dense model's attention layer after its 4096-token prompt
        dict(name="decode dense-4b 4k", op=DECODE, batch=1, t_lo=4096, t_hi=4096, window=0, sinks=0, nq=16, nkv=4, hd=128, page=128),
        # the MoE model's layer, eight sequences of ragged contexts
        dict(name="decode moe b8 ragged", op=DECODE, batch=8, t_lo=1024, t_hi=16384, window=0, sinks=0, nq=16, nkv=2, hd=256, page=128),
        # 64 long conversations that keep 4 first tokens and the last 1024
        dict(name="decode dense-4b b64 window", op=DECODE, batch=64, t_lo=500, t_hi=32768, window=1024, sinks=4, nq=16, nkv=4, hd=128,
             page=128),
        # eight very long contexts of the dense model, odd lengths: bandwidth
        dict(name="decode dense-4b b8 128k", op=DECODE, batch=8, t_lo=120001, t_hi=131000, window=0, sinks=0, nq=16, nkv=4, hd=128,
             page=128),
        # the tiny model's whole prompt
        dict(name="prompt tiny", op=PROMPT, batch=1, t_lo=0, t_hi=0, n_lo=37, n_hi=37, window=0, sinks=0, nq=4, nkv=2, hd=64, page=128),
        # the next short turns of eight conversations over their long contexts, few rows each
        dict(name="prompt moe b8 short turns", op=PROMPT, batch=8, t_lo=1024, t_hi=16384, n_lo=1, n_hi=24, window=0, sinks=0, nq=16,
             nkv=2, hd=256, page=128),
        # the third 2048-token chunk of a prompt of the dense model
        dict(name="prompt dense-4b 2048 at 4k", op=PROMPT, batch=1, t_lo=4096, t_hi=4096, n_lo=2048, n_hi=2048, window=0, sinks=0,
             nq=16, nkv=4, hd=128, page=128),
        # chunks of four long prompts under a window with sinks
        dict(name="prompt dense-4b b4 window", op=PROMPT, batch=4, t_lo=8000, t_hi=30000, n_lo=700, n_hi=2048, window=4096, sinks=4,
             nq=16, nkv=4, hd=128, page=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice([APPEND, DECODE, DECODE, PROMPT, PROMPT])
    hd = rng.choice([64, 128, 256])
    nkv = rng.choice([1, 2, 4, 8])
    nq = nkv * rng.choice([1, 2, 4, 8])
    c = dict(op=op, nq=nq, nkv=nkv, hd=hd, page=rng.choice([16, 64, 128, 128, 128, 208]))
    if op == APPEND:
        c["batch"] = rng.randint(1, 16)
        # at most the values of the largest listed case
        n_hi = _log_int(rng, 1, 4 * 2048 * 4 * 128 // (c["batch"] * nkv * hd))
        t_hi = rng.randint(0, 32768)
        return c | dict(t_lo=rng.randint(0, t_hi), t_hi=t_hi, n_lo=rng.randint(0, n_hi), n_hi=n_hi)
    if op == DECODE:
        c["batch"] = _log_int(rng, 1, 128)
        c["window"] = rng.choice([0, 0, _log_int(rng, 1, 8192)])
        c["sinks"] = rng.choice([0, 1, 4, 16, 100])
        rows = 8 * 4 * 128 * 120000 // (c["batch"] * nkv * hd)
        top = min(131000, rows)
        t_hi = _log_int(rng, 1, top)
        return c | dict(t_lo=rng.randint(0, t_hi), t_hi=t_hi)
    c["batch"] = rng.randint(1, 8)
    n_hi = _log_int(rng, 1, max(1, 2048 // c["batch"]))
    # the scores of the plain form: at most those of the largest listed case
    c["window"] = rng.choice([0, 0, _log_int(rng, 1, 4096)])
    c["sinks"] = rng.choice([0, 1, 4, 16, 100])
    top = max(1, min(32768, 16 * 2048 * 4096 * 128 // (c["batch"] * n_hi * nq * hd)))
    t_hi = rng.randint(0, top)
    return c | dict(t_lo=rng.randint(0, t_hi), t_hi=t_hi, n_lo=rng.randint(0, n_hi), n_hi=n_hi)


# ------------------------------------------------------------------ inputs
def _quantise(x):
    """Codes (int8, of x's shape [..., 16, hd]) and FP32 scales [...] of whole blocks of FP32 values that bf16 holds."""
    a = x.abs().amax((-2, -1))
    bad, small = ~torch.isfinite(a), a < 2.0 ** -100
    top = torch.full_like(a, 127.0)  # (a tensor: one correctly rounded division)
    inv = torch.where(small | bad, torch.zeros_like(a), top / a)
    c = torch.round(x * inv[..., None, None]).clamp(-127, 127)
    c = torch.where((small | bad)[..., None, None], torch.zeros_like(c), c)
    s = torch.where(bad, torch.full_like(a, math.nan), torch.where(small, torch.zeros_like(a), a / top))
    return c.to(torch.int8), s


def _rope_table(cap, hd):
    i = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
    ang = torch.arange(cap, device="cuda", dtype=torch.float64)[:, None] * torch.exp(-2 * i / hd * math.log(1e4))
    return torch.stack([ang.cos(), ang.sin()], -1).float()


def _lengths(case):
    """Each sequence's length before the call and its new rows: of the case alone, as the outputs' shapes go by them."""
    op, B = case["op"], case["batch"]
    rng = random.Random("%s %d %d %d" % (op, B, case["t_lo"], case["t_hi"]))
    lens = [case["t_hi"]] + [rng.randint(case["t_lo"], case["t_hi"]) for _ in range(B - 1)]
    if op == DECODE:
        return lens, [1] * B
    n = [case["n_hi"]] + [rng.randint(case["n_lo"], case["n_hi"]) for _ in range(B - 1)]
    if op == APPEND:
        # a chunk begins or ends at a block's border, so that a second pass finds the tail that the first found
        n = [k if t % BLOCK == 0 or (t + k) % BLOCK == 0 else max(0, -(-k // BLOCK) * BLOCK - t % BLOCK) for t, k in zip(lens, n)]
    return lens, n


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    st = dict(case)
    op, B, page = case["op"], case["batch"], case["page"]
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    lens, n = (torch.tensor(x, device="cuda") for x in _lengths(case))
    ends = lens + n
    rows = int(n.sum())
    st["rows"] = rows
    st["len"] = lens.to(torch.int32)
    st["row_start"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
    cap_pages = (int(ends.max()) + page) // page
    st["cap"] = cap = cap_pages * page
    # pages: those that a query of this call sees, or that it writes; a program gives the others back to the pool
    first = torch.arange(cap_pages, device="cuda") * page
    need = first[None] < ends[:, None]
    if op == APPEND:
        need &= first[None] + page > lens[:, None] // BLOCK * BLOCK
    elif case["window"]:
        need &= (first[None] + page > (lens - case["window"] + 1)[:, None]) | (first[None] < case["sinks"])
    need |= (ends[:, None] - 1) // page == torch.arange(cap_pages, device="cuda")[None]
    need[:, 0] |= True
    used = int(need.sum())
    st["pool"] = pool = used + 3
    ids = torch.randperm(pool, generator=g, device="cuda")[:used]
    table = torch.full((B, cap_pages), -1, device="cuda", dtype=torch.int64)
    table[need] = ids
    st["table"] = table.to(torch.int32)
    # closed blocks of normal k and v vectors
    bpp = page // BLOCK
    for name in ("K", "V"):
        codes = torch.empty((pool, nkv, page, hd), dtype=torch.int8, device="cuda")
        scales = torch.empty((pool, nkv, bpp), device="cuda")
        step = max(1, (1 << 26) // (nkv * page * hd))
        for p in range(0, pool, step):
            k = min(pool, p + step) - p
            x = torch.randn((k, nkv, bpp, BLOCK, hd), generator=g, device="cuda").bfloat16().float()
            c, s = _quantise(x)
            codes[p:p + k], scales[p:p + k] = c.view(k, nkv, page, hd), s
        st[name], st[name + "s"] = codes, scales
    st["tail"] = torch.randn((B, 2, nkv, BLOCK, hd), generator=g, device="cuda").bfloat16()
    st["y"] = torch.randn((max(rows, 1), (nq + 2 * nkv) * hd), generator=g, device="cuda")
    st["y"][:, :nq * hd] *= 1.5
    st["rope"] = _rope_table(cap, hd)
    if op == PROMPT:
        # per row: its sequence and its place there; a scheduler has both
        st["seq"] = torch.repeat_interleave(torch.arange(B, device="cuda"), n)
        st["at"] = torch.arange(rows, device="cuda") - st["row_start"].long()[st["seq"]]
        st["n_max"] = int(n.max())
    elif op == APPEND:
        st["seq"] = torch.repeat_interleave(torch.arange(B, device="cuda"), n)
        st["at"] = torch.arange(rows, device="cuda") - st["row_start"].long()[st["seq"]]
        # the blocks that the new rows touch, one after the other: their sequence and number
        lo, hi = lens // BLOCK, torch.where(n > 0, (ends - 1) // BLOCK + 1, lens // BLOCK)
        st["blk_seq"] = torch.repeat_interleave(torch.arange(B, device="cuda"), hi - lo)
        start = torch.cat([lo.new_zeros(1), (hi - lo).cumsum(0)])
        st["blk"] = torch.arange(int(start[-1]), device="cuda") - start[st["blk_seq"]] + lo[st["blk_seq"]]
        st["blk_start"] = start
    if op != APPEND:
        # what the queries can see at most, as a list of blocks for each sequence (-1: none)
        w, s = case["window"], case["sinks"]
        nb = (ends - 1).clamp(min=0) // BLOCK + 1
        lo = ((lens - w + 1).clamp(min=0) // BLOCK) if w else torch.zeros_like(lens)
        ns = torch.minimum(lo, torch.full_like(lo, (s + BLOCK - 1) // BLOCK))
        width = int((ns + nb - lo).max())
        i = torch.arange(width, device="cuda")[None]
        st["view"] = torch.where(i < ns[:, None], i, i - ns[:, None] + lo[:, None])
        st["view"] = torch.where(i < (ns + nb - lo)[:, None], st["view"], torch.full_like(st["view"], -1))
        st["end"] = ends
    if own:
        from bandwidth_bound_hybrid_gb300 import capi
        st["kv"] = capi.hy_kv_p8(st["K"].data_ptr(), st["V"].data_ptr(), st["Ks"].data_ptr(), st["Vs"].data_ptr(),
                                 st["K"].stride(0), st["Ks"].stride(0), page, pool, st["tail"].data_ptr(), st["tail"].stride(0) * 2,
                                 st["table"].data_ptr(), cap_pages)
        if op != APPEND:
            size = (capi.lib().hy_op_attention_p8_workspace(B, nq, nkv, hd) if op == DECODE else
                    capi.lib().hy_op_attention_p8_prompt_workspace(rows, B, nq, nkv, hd))
            st["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms
def _rotated(st, x, pos):
    """FP32 vectors [rows, heads, hd] rotated for their positions [rows]."""
    h = st["hd"] // 2
    cs = st["rope"][pos]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    x0, x1 = x[..., :h], x[..., h:]
    return torch.cat([x0 * c - x1 * s, x1 * c + x0 * s], -1)


def _new_kv(st, y, pos):
    """bf16 values (as FP32) of the rows' k and v: [rows, 2, nkv, hd]."""
    nq, nkv = st["nq"], st["nkv"]
    y = y.unflatten(-1, (-1, st["hd"]))
    return torch.stack([_rotated(st, y[:, nq:nq + nkv], pos), y[:, nq + nkv:]], 1).bfloat16().float()


def _close(st, b, blk, x):
    """Blocks x [m, 2, nkv, 16, hd] written as block blk[m] of sequence b[m]; their values."""
    codes, scales = _quantise(x)
    bpp = st["page"] // BLOCK
    pg, at = st["table"][b, blk // bpp].long(), blk % bpp
    row = (at * BLOCK)[:, None] + torch.arange(BLOCK, device="cuda")
    for w, name in ((0, "K"), (1, "V")):
        st[name][pg[:, None], :, row] = codes[:, w].transpose(1, 2)
        st[name + "s"][pg, :, at] = scales[:, w]
    return codes.float() * scales[..., None, None]


def _plain_append(st):
    b, at = st["seq"], st["at"]
    pos = st["len"].long()[b] + at
    new = _new_kv(st, st["y"][:st["rows"]], pos)
    # the touched blocks, rows before the new ones from the tail
    m, e = st["blk_seq"], st["blk"]
    x = torch.where((e == st["len"].long()[m] // BLOCK)[:, None, None, None, None], st["tail"][m].float(),
                    torch.zeros((), device="cuda"))
    slot = st["blk_start"][b] + pos // BLOCK - st["len"].long()[b] // BLOCK
    x[slot, :, :, pos % BLOCK] = new
    end = st["len"].long() + st["row_start"][1:].long() - st["row_start"][:-1].long()
    whole = (e + 1) * BLOCK <= end[m]
    val = x.clone()
    val[whole] = _close(st, m[whole], e[whole], x[whole])
    # a block that stays open holds the tail's new rows
    last = pos // BLOCK == end[b] // BLOCK
    st["tail"][b[last], :, :, pos[last] % BLOCK] = new[last].bfloat16()
    return {"kv_new": val[slot, :, :, pos % BLOCK], "tail": st["tail"]}


def _held(st, tail):
    """Values of the blocks of st["view"]: K and V [B, nkv, width * 16, hd] and the positions [B, width * 16] (-1: none)."""
    view = st["view"]
    bpp = st["page"] // BLOCK
    pg = st["table"].gather(1, (view.clamp(min=0) // bpp)).long().clamp(min=0)
    at = view.clamp(min=0) % bpp
    is_tail = (view == (st["end"] // BLOCK)[:, None])[:, :, None, None, None]
    out = []
    for w, name in ((0, "K"), (1, "V")):
        codes = st[name].view(st["pool"], st["nkv"], bpp, BLOCK, st["hd"])[pg, :, at]  # [B, width, nkv, 16, hd]
        x = codes.float() * st[name + "s"][pg, :, at][..., None, None]
        x = torch.where(is_tail, tail[:, w].float()[:, None], x)
        out.append(x.transpose(1, 2).flatten(2, 3))
    pos = view[:, :, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    pos = torch.where(view[:, :, None] >= 0, pos, torch.full_like(pos, -1)).flatten(1)
    return out[0], out[1], pos


def _attend(st, q, t, K, V, pos):
    """q [B, n, nq, hd] at positions t [B, n] (-1: no query) over K, V [B, nkv, m, hd] at positions pos [B, m]: [B, n, nq, hd]."""
    B, n, nq, hd = q.shape
    nkv, m = st["nkv"], K.shape[2]
    q = q.unflatten(2, (nkv, nq // nkv)).permute(0, 2, 1, 3, 4).reshape(B, nkv, n * (nq // nkv), hd)
    s = torch.matmul(q, K.transpose(-1, -2)).mul_(1 / math.sqrt(hd)).view(B, nkv, n, nq // nkv, m)
    u = pos[:, None, :]
    seen = (u >= 0) & (u <= t[:, :, None])
    if st["window"]:
        seen &= (u < st["sinks"]) | (u > t[:, :, None] - st["window"])
    s.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    s = torch.exp_(s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30)))
    o = torch.matmul(s.view(B, nkv, -1, m), V) / s.sum(-1).view(B, nkv, -1, 1).clamp(min=1e-30)
    return o.view(B, nkv, n, nq // nkv, hd).permute(0, 2, 1, 3, 4).reshape(B, n, nq, hd)


def _plain_decode(st):
    B, nq, hd = st["batch"], st["nq"], st["hd"]
    T = st["len"].long()
    b = torch.arange(B, device="cuda")
    new = _new_kv(st, st["y"], T)
    full = st["tail"].float()
    full[b, :, :, T % BLOCK] = new
    closes = T % BLOCK == BLOCK - 1
    val = new.clone()
    val[closes] = _close(st, b[closes], (T // BLOCK)[closes], full[closes])[:, :, :, BLOCK - 1]
    # the tail keeps a row of the open block; that of a block that closes goes to the page alone
    st["tail"][b[~closes], :, :, (T % BLOCK)[~closes]] = new[~closes].bfloat16()
    K, V, pos = _held(st, st["tail"])
    q = _rotated(st, st["y"].unflatten(-1, (-1, hd))[:, :nq], T)
    o = _attend(st, q[:, None], T[:, None], K, V, pos)
    return {"o": o.reshape(B, nq * hd), "kv_new": val, "tail": st["tail"]}


def _plain_prompt(st):
    B, nq, hd, rows = st["batch"], st["nq"], st["hd"], st["rows"]
    b, at = st["seq"], st["at"]
    pos = st["len"].long()[b] + at
    q = torch.zeros((B, st["n_max"], nq, hd), device="cuda")
    t = torch.full((B, st["n_max"]), -1, device="cuda", dtype=torch.int64)
    q[b, at] = _rotated(st, st["y"][:rows].unflatten(-1, (-1, hd))[:, :nq], pos)
    t[b, at] = pos
    K, V, held = _held(st, st["tail"])
    return {"o": _attend(st, q, t, K, V, held)[b, at].reshape(rows, nq * hd)}


# ------------------------------------------------------------------ the framework's calls
def _own(st):
    import ctypes

    from bandwidth_bound_hybrid_gb300 import capi
    L = capi.lib()
    op, B, nq, nkv, hd = st["op"], st["batch"], st["nq"], st["nkv"], st["hd"]
    stream = torch.cuda.current_stream().cuda_stream
    y, kv = st["y"], ctypes.byref(st["kv"])
    if op == APPEND:
        new = torch.empty((st["rows"], 2, nkv, hd), device="cuda")
        capi.check(L.hy_op_kv_append_p8(y.data_ptr(), y.stride(0), st["rows"], B, st["row_start"].data_ptr(), kv, nq, nkv, hd,
                                        st["len"].data_ptr(), st["rope"].data_ptr(), new.data_ptr(), stream), "hy_op_kv_append_p8")
        return {"kv_new": new, "tail": st["tail"]}
    if op == DECODE:
        o = torch.empty((B, nq * hd), device="cuda")
        new = torch.empty((B, 2, nkv, hd), device="cuda")
        capi.check(L.hy_op_attention_p8(y.data_ptr(), y.stride(0), B, kv, nq, nkv, hd, st["window"], st["sinks"],
                                        st["len"].data_ptr(), st["rope"].data_ptr(), o.data_ptr(), nq * hd, new.data_ptr(),
                                        st["ws"].data_ptr(), stream), "hy_op_attention_p8")
        return {"o": o, "kv_new": new, "tail": st["tail"]}
    o = torch.empty((st["rows"], nq * hd), device="cuda")
    capi.check(L.hy_op_attention_p8_prompt(y.data_ptr(), y.stride(0), st["rows"], B, st["row_start"].data_ptr(), kv, nq, nkv, hd,
                                           st["window"], st["sinks"], st["len"].data_ptr(), st["rope"].data_ptr(), o.data_ptr(),
                                           nq * hd, st["ws"].data_ptr(), stream), "hy_op_attention_p8_prompt")
    return {"o": o}


def run(state):
    if own:
        return _own(state)
    if state["op"] == APPEND:
        return _plain_append(state)
    if state["op"] == DECODE:
        return _plain_decode(state)
    return _plain_prompt(state)


# ------------------------------------------------------------------ floors
def work(case):
    op, nq, nkv, hd = case["op"], case["nq"], case["nkv"], case["hd"]
    w, sinks = case.get("window", 0), case.get("sinks", 0)
    row = nkv * 2 * (hd + 4 / BLOCK)  # codes and scales of a position
    sizes = [(t, k) for t, k in zip(*_lengths(case)) if k]
    n = sum(k for _, k in sizes)

    def seen(t):  # positions that a query at t sees
        return min(t + 1, w) + min(sinks, max(0, t + 1 - w)) if w else t + 1

    # open rows that are read, and new ones that are written, in bf16
    tails = sum(nkv * 2 * hd * 2 * ((t % BLOCK if op != PROMPT else (t + k) % BLOCK) + (0 if op == PROMPT else min(k, (t + k) % BLOCK)))
                for t, k in sizes)
    if op == APPEND:
        return {"bytes": n * (nkv * 2 * 8 * hd + row + 4 * hd) + tails, "flops": 8.0 * n * nkv * hd}
    pairs = sum(sum(seen(t + i) for i in range(k)) for t, k in sizes)
    flops = 4.0 * nq * hd * pairs
    if op == DECODE:
        return {"bytes": pairs * row + tails + n * (4 * (2 * nq + 2 * nkv) * hd + 4 * hd + 2 * nkv * hd * 4), "flops": flops}
    kept = sum(min(t + k, w + k - 1 + sinks) if w else t + k for t, k in sizes)
    return {"bytes": kept * row + tails + n * (8 * nq * hd + 4 * hd), "flops": flops}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, B, nq, nkv, hd, page = case["op"], case["batch"], case["nq"], case["nkv"], case["hd"], case["page"]
    G, half = nq // nkv, hd // 2
    lens, starts, table = st["len"].tolist(), st["row_start"].tolist(), st["table"].tolist()
    y = st["y"].view(-1, nq + 2 * nkv, hd)

    def stored(rows, T):
        """The bf16 rows [2, nkv, n, hd] that the format holds of projection rows at positions T on (FP32 operations)."""
        n = rows.shape[0]
        cs = st["rope"][T:T + n]
        c, s = cs[None, :, :, 0], cs[None, :, :, 1]
        k, v = rows[:, nq:nq + nkv].transpose(0, 1), rows[:, nq + nkv:].transpose(0, 1)
        k0, k1 = k[..., :half], k[..., half:]
        k = torch.cat([(k0 * c) - (k1 * s), (k1 * c) + (k0 * s)], -1)
        return torch.stack([k, v]).bfloat16()

    def closed(block):
        """The values of a block [16, hd] of bf16 rows once it is closed."""
        top = float(block.abs().max())
        if top < 2.0 ** -100:
            return torch.zeros((BLOCK, hd), dtype=torch.float64, device="cuda")
        a = block.float().abs().max()
        code = (block.float() * (torch.full_like(a, 127.0) / a)).round().clamp(-127, 127)
        return code.double() * (a / torch.full_like(a, 127.0)).double()

    def values(before, new, T):
        """The rows [2, nkv, n, hd] at positions T on as they are held after the append; `before`: the open block's rows."""
        n = new.shape[2]
        out = new.double()
        for j in range(T // BLOCK, (T + n) // BLOCK):  # blocks that are whole now
            lo, hi = j * BLOCK - T, j * BLOCK - T + BLOCK
            whole = new[:, :, lo:hi] if lo >= 0 else torch.cat([before[:, :, :-lo], new[:, :, :hi]], 2)
            for w in range(2):
                for h in range(nkv):
                    out[w, h, max(lo, 0):hi] = closed(whole[w, h])[max(0, -lo):]
        return out

    if op == APPEND:
        parts, tail = [], st["tail"].double()
        for b in range(B):
            T, rows = lens[b], y[starts[b]:starts[b + 1]]
            new = stored(rows, T)
            parts.append(values(st["tail"][b][:, :, :T % BLOCK], new, T).permute(2, 0, 1, 3))
            for i in range(rows.shape[0]):
                if (T + i) // BLOCK == (T + rows.shape[0]) // BLOCK:
                    tail[b, :, :, (T + i) % BLOCK] = new[:, :, i].double()
        return {"kv_new": torch.cat(parts), "tail": tail}

    def cached(name, b, h, n):
        """The values of positions [0, n) (whole blocks) in the pages; NaN where the sequence has no page."""
        pg = st["table"][b, :(n + page - 1) // page].long()
        x = st[name][pg.clamp(min=0), h].double().view(-1, page // BLOCK, BLOCK, hd)
        x = x * st[name + "s"][pg.clamp(min=0), h].double()[:, :, None, None]
        return torch.where(pg[:, None, None, None] < 0, math.nan, x).view(-1, hd)[:n]

    w, sinks = case["window"], case["sinks"]
    o = torch.zeros((y.shape[0] if op == DECODE else starts[-1], nq, hd), dtype=torch.float64, device="cuda")
    tail, new_out = st["tail"].double(), []
    for b in range(B):
        T = lens[b]
        rows = y[b:b + 1] if op == DECODE else y[starts[b]:starts[b + 1]]
        n = rows.shape[0]
        if n == 0:
            continue
        r0 = b if op == DECODE else starts[b]
        if op == DECODE:
            new = stored(rows, T)
            val = values(st["tail"][b][:, :, :T % BLOCK], new, T)
            new_out.append(val[:, :, 0])
            if T % BLOCK < BLOCK - 1:
                tail[b, :, :, T % BLOCK] = new[:, :, 0].double()
        t = torch.arange(T, T + n, device="cuda")
        end = T + n
        u = torch.arange(end, device="cuda")
        seen = u[None] <= t[:, None]
        if w:
            seen &= (u[None] < sinks) | (u[None] > t[:, None] - w)
        keep = seen.any(0)
        u, seen = u[keep], seen[:, keep]
        cd, sd = st["rope"][T:end, :, 0].double(), st["rope"][T:end, :, 1].double()
        for h in range(nkv):
            kvs = []
            for i, name in ((0, "K"), (1, "V")):
                x = torch.empty((end, hd), dtype=torch.float64, device="cuda")
                m = end // BLOCK * BLOCK
                x[:m] = cached(name, b, h, m)
                x[m:] = tail[b, i, h, :end - m]
                if op == DECODE and m == end:  # the row that closes its block: as it is held from now on
                    before = st["tail"][b, i, h, :BLOCK - 1]
                    x[end - BLOCK:] = closed(torch.cat([before, new[i, h]]))
                kvs.append(x[keep])
            for j in range(h * G, h * G + G):
                q = rows[:, j].double()
                q = torch.cat([q[:, :half] * cd - q[:, half:] * sd, q[:, half:] * cd + q[:, :half] * sd], -1)
                a = q @ kvs[0].T / math.sqrt(hd)
                a = torch.softmax(torch.where(seen, a, torch.full_like(a, -math.inf)), -1)
                o[r0:r0 + n, j] = a @ kvs[1]
    if op == DECODE:
        return {"o": o.flatten(1), "kv_new": torch.stack(new_out), "tail": tail}
    return {"o": o.flatten(1)}
