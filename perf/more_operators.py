"""Timing cases of the serving operators around the quantised products: the residual's addition with
its RMS norm, rotation and int8 output; pages taken and given back on the GPU; the append into a
cache held in 4 bits, and attention over that cache.

Every case is one pass of one operator.  Where `own` is false `run` computes it with
elementary torch operations; where it is true it calls the package's kernels.  `exact` computes
the same from the definitions in 64 bits.

Definitions (fp32 unless said otherwise, one rounding to each output's type):

  norm      h = x + r, rounded to r's type;  f = fl32(1 / sqrt(mean(h^2) + eps)), the mean and the
            root in 64 bits;  y = fl32(fl32(h f) (w + offset));  each block of 256 of y through the
            Hadamard transform by butterflies of span 1, 2, .. 128, then 1/16;  s = max|.| / 127 of a
            token, codes clamp(rint(. / s), -127, 127), 0 where s = 0
  assign    sequence b grows from seq_lens[b] by new_tokens[b]; the pages that it lacks come off the
            free list's end, sequence by sequence (-1 where it has run out).  Out: the page table's
            new entries, offsets and lengths, position and slot (page * page size + place) of each
            new token (0 and -1 behind the last), the list's new length, the pages that were missing
  release   sequence b shrinks to keep_lens[b]; the pages behind go back to the list, the last of the
            last sequence first, so that assigning again hands out the same ones
  append    16 consecutive values of a token's head share a scale sc(byte) * unit: with t = max|x| /
            fl32(6 unit), byte is the nearest of 1 .. 255 to t, ties to even, sc(b) = b below 16, else
            (16 + b % 16) 2^(b / 16 - 1); a value is the nearest of +-{0, .5, 1, 1.5, 2, 3, 4, 6} to
            fl32(x / fl32(sc unit)), ties to the even code, two codes a byte, the first one low
  attn      token i of the n new ones of a sequence of length len (new ones included) sits at position
            p = len - n + i and sees positions max(0, p - window + 1) .. p (all of 0 .. len - 1 where
            the case is not causal); softmax(scale q.k) v over them
"""
import math
import random

import torch

own = False

EPS = 1e-6
UNIT = 2.0 ** -14


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one generated token between two layers of the hybrid decoder (hidden size 5120): latency
        dict(name="norm 1 token", op="norm", tokens=1, k=5120, x="f32", r="bf16", y=""),
        # a served batch's tokens; the normed values also go to projections that are not quantised
        dict(name="norm 61 tokens + normed", op="norm", tokens=61, k=5120, x="bf16", r="f32", y="bf16"),
        # a long prompt
        dict(name="norm 8192 tokens", op="norm", tokens=8192, k=5120, x="f32", r="bf16", y=""),
        # a decode step of a served batch: most sequences stay inside their last page
        dict(name="assign 61 x 1", op="assign", seqs=61, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=4000, page=64, ragged=31),
        # prompts and chunks of prompts of many requests that arrive together, small pages
        dict(name="assign 700 ragged", op="assign", seqs=700, new_lo=0, new_hi=400, ctx_lo=0, ctx_hi=3000, page=16, ragged=32),
        # requests that end, and drafts that were refused, in a large batch
        dict(name="release 1021", op="release", seqs=1021, new_lo=0, new_hi=500, ctx_lo=0, ctx_hi=2000, page=16, ragged=33),
        # one new token for each of 61 sequences
        dict(name="append 61 x 1", op="append", seqs=61, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=4000, hkv=4, d=256, page=64,
             dtype="bf16", ragged=41),
        # three prompts, the later chunks of which continue partly filled pages
        dict(name="append 3 x 2731", op="append", seqs=3, new_lo=2731, new_hi=2731, ctx_lo=0, ctx_hi=500, hkv=4, d=256,
             page=64, dtype="bf16", ragged=42),
        # decode of one short conversation: latency
        dict(name="decode 1 x 777", op="attn", seqs=1, new_lo=1, new_hi=1, ctx_lo=776, ctx_hi=776, hq=24, hkv=4, d=256,
             page=16, window=0, causal=True, dtype="bf16", ragged=51),
        # decode far into the model's context of 262,144 tokens, what a cache in 4 bits is for
        dict(name="decode 4 long", op="attn", seqs=4, new_lo=1, new_hi=1, ctx_lo=90001, ctx_hi=131072, hq=24, hkv=4, d=256,
             page=128, window=0, causal=True, dtype="bf16", ragged=52),
        # a sliding window, one cache head for each query head, heads of 64, fp32, chunks of odd sizes
        dict(name="window 7 ragged fp32", op="attn", seqs=7, new_lo=1, new_hi=700, ctx_lo=0, ctx_hi=2000, hq=16, hkv=16, d=64,
             page=16, window=512, causal=True, dtype="f32", ragged=53),
        # chunks of two prompts that already have a context
        dict(name="prefill 2 x 2048 + 14k", op="attn", seqs=2, new_lo=1900, new_hi=2048, ctx_lo=14000, ctx_hi=14500, hq=24,
             hkv=4, d=256, page=64, window=0, causal=True, dtype="bf16", ragged=54),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 5, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 6, 7, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.randrange(1 << 30)
    op = rng.choice(["norm", "norm", "assign", "release", "append", "append", "attn", "attn", "attn", "attn"])
    if op == "norm":
        k = 256 * _log_int(rng, 1, 80)
        return dict(op="norm", tokens=_log_int(rng, 1, 8192 * 5120 // max(5120, k)), k=k, x=rng.choice(["f32", "bf16"]),
                    r=rng.choice(["f32", "bf16"]), y=rng.choice(["", "", "f32", "bf16"]))
    if op in ("assign", "release"):
        seqs = _log_int(rng, 1, 3000)
        hi = _log_int(rng, 1, max(2, 200000 // seqs))
        return dict(op=op, seqs=seqs, new_lo=rng.randint(0, hi), new_hi=hi, ctx_lo=0, ctx_hi=_log_int(rng, 1, 4000), page=page,
                    ragged=ragged)
    if op == "append":
        seqs = _log_int(rng, 1, 100)
        hi = _log_int(rng, 1, max(2, 8192 // seqs))
        return dict(op="append", seqs=seqs, new_lo=rng.randint(1, hi), new_hi=hi, ctx_lo=0, ctx_hi=_log_int(rng, 1, 3000),
                    hkv=hkv, d=d, page=page, dtype=dtype, ragged=ragged)
    if rng.random() < 0.6:  # decode, few new tokens
        seqs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 5)
        ctx = _log_int(rng, 30, 262144 // seqs)
    else:                   # prompts and their chunks
        seqs = _log_int(rng, 1, 8)
        hi = _log_int(rng, 6, 3800 // seqs)
        ctx = _log_int(rng, 1, 12000)
    return dict(op="attn", seqs=seqs, new_lo=rng.randint(1, hi), new_hi=hi, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx, hq=hq,
                hkv=hkv, d=d, page=page, window=rng.choice([0, 0, 0, _log_int(rng, 16, 4096)]), causal=rng.random() < 0.85,
                dtype=dtype, ragged=ragged)


def _lengths(case):
    """The host's view of a batch: new tokens and lengths (new ones included) of each sequence."""
    r = random.Random(case["ragged"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    old = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["seqs"])]
    return new, [n + o for n, o in zip(new, old)]


def _seen(case):
    """(query, key) pairs that attention looks at, and cache tokens that any query of a sequence sees."""
    pairs = tokens = 0
    for n, length in zip(*_lengths(case)):
        first = length - n
        if not case["causal"]:
            pairs += n * length
            tokens += length
        elif case["window"]:
            pairs += sum(min(case["window"], first + i + 1) for i in range(n))
            tokens += length - max(0, first - case["window"] + 1)
        else:
            pairs += n * first + n * (n + 1) // 2
            tokens += length
    return pairs, tokens


def _size(name):
    return {"": 0, "bf16": 2, "f32": 4}[name]


def _page_moves(case):
    """Pages that a batch's new tokens take, or give back."""
    p = case["page"]
    return sum(-(-length // p) - -(-(length - n) // p) for n, length in zip(*_lengths(case)))


def work(case):
    if case["op"] == "norm":
        values = case["tokens"] * case["k"]
        return {"bytes": values * (_size(case["x"]) + 2 * _size(case["r"]) + _size(case["y"]) + 1) + 4 * case["tokens"] + 4 * case["k"],
                "flops": values * 17}
    new, lens = _lengths(case)
    if case["op"] == "assign":  # lengths, offsets and tokens of a sequence, a page twice, a token's position and slot
        return {"bytes": 16 * case["seqs"] + 8 * _page_moves(case) + 12 * sum(new), "flops": sum(new)}
    if case["op"] == "release":
        return {"bytes": 12 * case["seqs"] + 8 * _page_moves(case), "flops": case["seqs"]}
    d, hkv = case["d"], case["hkv"]
    row = hkv * (d // 2 + d // 16)  # bytes of a token's keys or values in the cache
    if case["op"] == "append":
        return {"bytes": 2 * sum(new) * (hkv * d * _size(case["dtype"]) + row) + 8 * sum(new), "flops": 8 * sum(new) * hkv * d}
    pairs, tokens = _seen(case)
    return {"bytes": 2 * sum(new) * case["hq"] * d * _size(case["dtype"]) + 2 * tokens * row,
            "flops": 4 * pairs * case["hq"] * d}


# ----------------------------------------------------------------------------- inputs

def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _batch(case, gen):
    """A batch whose pages are all there, in random order: table, offsets of the new tokens, lengths."""
    new, lens = _lengths(case)
    page = case["page"]
    width = max(max(-(-length // page) for length in lens), 1)
    counts = torch.tensor([-(-length // page) for length in lens], device="cuda")
    pages = max(1, int(sum(-(-length // page) for length in lens)))
    order = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    table = torch.zeros((case["seqs"], width), dtype=torch.int32, device="cuda")
    there = torch.arange(width, device="cuda")[None, :] < counts[:, None]
    table[there] = order[:int(counts.sum())]
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    return dict(table=table, cu=torch.tensor(off, dtype=torch.int32, device="cuda"),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), pages=pages, new=new, lengths=lens)


def _filled(case, pages, gen, spread):
    """Pages of keys or values held in 4 bits: normal values, some channels wide."""
    hkv, page, d = case["hkv"], case["page"], case["d"]
    wide = 1.0 + 3.0 * (torch.rand((1, hkv, 1, d), generator=gen, device="cuda") > 0.95)
    codes = torch.empty((pages, hkv, page, d // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, hkv, page, d // 16), dtype=torch.uint8, device="cuda")
    unit = torch.full((hkv,), UNIT, device="cuda")
    step = max(1, (1 << 26) // (hkv * page * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn((n, hkv, page, d), generator=gen, device="cuda") * wide * spread
        codes[p:p + n], scales[p:p + n] = _quantise4(x, unit[None, :, None, None])
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    state = dict(case=case)
    if case["op"] == "norm":
        m, k = case["tokens"], case["k"]
        # a residual stream: some channels far wider than the others
        wide = 1.0 + 30.0 * (torch.rand(k, generator=gen, device="cuda") > 0.995)
        state |= dict(x=(rand(m, k) * 0.5).to(_type(case["x"])), r=(rand(m, k) * wide).to(_type(case["r"])), w=rand(k) * 0.2)
        return state
    if case["op"] in ("assign", "release"):
        new, lens = _lengths(case)
        b = _batch(case, gen)
        old = torch.tensor([length - n for n, length in zip(new, lens)], dtype=torch.int32, device="cuda")
        page = case["page"]
        have = (-(-old.long() // page))[:, None]
        mine = torch.arange(b["table"].shape[1], device="cuda")[None, :] < have
        spare = 17
        if case["op"] == "assign":
            # the pages of the old tokens are in the table, the others on the free list with some to spare
            taken = torch.zeros(b["pages"], dtype=torch.bool, device="cuda")
            taken[b["table"][mine].long()] = True
            free = torch.nonzero(~taken)[:, 0].to(torch.int32)
            free = free[torch.randperm(free.numel(), generator=gen, device="cuda")]
            free = torch.cat([torch.arange(b["pages"], b["pages"] + spare, dtype=torch.int32, device="cuda"), free])
            stack = torch.full((b["pages"] + spare,), -1, dtype=torch.int32, device="cuda")
            stack[:free.numel()] = free
            state |= dict(table=torch.where(mine, b["table"], 0), lens=old, stack=stack,
                          count=torch.tensor([free.numel()], dtype=torch.int32, device="cuda"),
                          new=torch.tensor(new, dtype=torch.int32, device="cuda"), tokens=sum(new) + 3)
        else:
            stack = torch.full((b["pages"] + spare,), -1, dtype=torch.int32, device="cuda")
            stack[:spare] = torch.arange(b["pages"], b["pages"] + spare, dtype=torch.int32, device="cuda")
            # an eighth of the requests end; the others give up what `new` says of their tokens
            ended = torch.rand(case["seqs"], generator=gen, device="cuda") < 0.125
            state |= dict(table=b["table"], lens=b["lens"], stack=stack, keep=torch.where(ended, 0, old).to(torch.int32),
                          count=torch.tensor([spare], dtype=torch.int32, device="cuda"))
        if own:
            from w4a8_codebook_gemm_amd import serving as S
            state["pages"] = S.Pages(state["table"], state["lens"], state["stack"], state["count"], page)
            if case["op"] == "assign":
                state["batch"] = S.Batch.empty(case["seqs"], state["tokens"])
        return state
    b = _batch(case, gen)
    m, d, hkv = sum(b["new"]), case["d"], case["hkv"]
    state |= dict(batch=b, unit=torch.full((hkv,), UNIT, device="cuda"))
    state["kc"], state["ks"] = _filled(case, b["pages"], gen, 1.0)
    state["vc"], vs = _filled(case, b["pages"], gen, 0.5)
    state["vs"] = vs.transpose(2, 3).contiguous()  # a group's scales of a page lie together
    if case["op"] == "append":
        # keys from the norm and rotation, values as a part of a projection's wider rows
        state |= dict(k=(rand(m, hkv, d) * 1.2).to(_type(case["dtype"])),
                      v=(rand(m, 2 * hkv, d) * 0.6).to(_type(case["dtype"]))[:, hkv:])
        _, _, page, slot = _places(state)
        state["slots"] = page * case["page"] + slot
    else:
        state |= dict(q=rand(m, case["hq"], d).to(_type(case["dtype"])), scale=d ** -0.5)
    if own:
        from w4a8_codebook_gemm_amd import attention as A
        from w4a8_codebook_gemm_amd import serving as S
        state["cache"] = S.KV4Cache(state["kc"], state["vc"], state["ks"], state["vs"], state["unit"], state["unit"])
        if case["op"] == "attn":
            state["seqs"] = A.Sequences(b["table"], b["cu"], b["lens"])
            state["workspace"] = S.kv4_attention_workspace(m, case["seqs"], case["hq"], hkv, d, device="cuda")
    return state


# ----------------------------------------------------------------------------- the plain forms

def _norm_plain(s):
    c = s["case"]
    m, k = s["x"].shape
    h = (s["x"].float() + s["r"].float()).to(_type(c["r"]))
    f = (1.0 / torch.sqrt(h.double().square().mean(-1, keepdim=True) + EPS)).float()
    y = h.float() * f * (s["w"] + 1.0)
    z = y
    for span in (1, 2, 4, 8, 16, 32, 64, 128):  # the transform's eight stages
        z = z.view(m, k // (2 * span), 2, span)
        z = torch.stack((z[:, :, 0] + z[:, :, 1], z[:, :, 0] - z[:, :, 1]), 2)
    z = z.view(m, k) * 0.0625
    top = z.abs().amax(-1)
    scale = top / torch.full_like(top, 127.0)
    codes = torch.where(scale[:, None] > 0, torch.round(z / scale[:, None]), 0).clamp(-127, 127).to(torch.int8)
    return h, codes, scale, y.to(_type(c["y"])) if c["y"] else None


def _assign_plain(s):
    page, b, tokens = s["case"]["page"], s["case"]["seqs"], s["tokens"]
    width = s["table"].shape[1]
    old, new, count = s["lens"].long(), s["new"].long(), s["count"].long()
    end = torch.cumsum(new, 0)
    cu = torch.cat((torch.zeros_like(end[:1]), end))
    have, need = (old + page - 1) // page, (old + new + page - 1) // page
    first = torch.cumsum(need - have, 0) - (need - have)
    entry = torch.arange(width, device="cuda")[None, :]
    fresh = (entry >= have[:, None]) & (entry < need[:, None])
    at = count - 1 - (first[:, None] + entry - have[:, None])
    s["table"].copy_(torch.where(fresh, torch.where(at >= 0, s["stack"][at.clamp(min=0, max=s["stack"].numel() - 1)], -1), s["table"]))
    token = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(end, token, right=True)
    real = seq < b
    seq = seq.clamp(max=b - 1)
    pos = old[seq] + token - cu[seq]
    got = s["table"].long()[seq, torch.where(real, pos // page, 0)]
    taken = (need - have).sum()
    return dict(table=s["table"], cu=cu.int(), lens=(old + new).int(), positions=torch.where(real, pos, 0).int(),
                slots=torch.where(real & (got >= 0), got * page + pos % page, -1),
                count=(count - taken).clamp(min=0).int(), missing=(taken - count).clamp(min=0).int())


def _release_plain(s):
    page = s["case"]["page"]
    width = s["table"].shape[1]
    old = s["lens"].long()
    keep = torch.minimum(s["keep"].long(), old)
    have, stay = (old + page - 1) // page, (keep + page - 1) // page
    entry = torch.arange(width, device="cuda")[None, :]
    gone = ((entry >= stay[:, None]) & (entry < have[:, None])).flatten()
    rank = torch.cumsum(gone, 0)
    spare = s["stack"].numel()  # a place behind the list, for the entries that stay
    place = torch.where(gone, (s["count"] + rank[-1] - rank).clamp(max=spare), spare)
    s["stack"].copy_(torch.cat((s["stack"], s["stack"][:1])).scatter_(0, place, s["table"].flatten())[:spare])
    return dict(stack=s["stack"], lens=keep.int(), count=(s["count"] + rank[-1]).int())


def _quantise4(x, unit):
    """Codes two a byte and scale bytes of x [..., d] in fp32; unit broadcasts against x."""
    g = x.unflatten(-1, (-1, 16))
    u = unit[..., None]
    t = g.abs().amax(-1, keepdim=True) / (u * 6.0)
    up = (torch.frexp(t)[1] - 5).clamp(min=0, max=14)           # t is 16 .. 32 steps of 2^up
    n = torch.round(t.clamp(max=1e9) * torch.exp2(-up.float()))  # to even
    byte = (up * 16 + n).clamp(1, 255)
    sc = torch.where(byte < 16, byte, (16 + byte % 16) * torch.exp2(torch.floor(byte / 16) - 1))
    y = g / (sc * u)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
            + 8 * torch.signbit(y).to(torch.uint8))
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte[..., 0].to(torch.uint8)


def _values4(codes, scales, unit):
    """The values that codes [..., d / 2] and scales [..., d / 16] stand for, in unit's type."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=unit.dtype, device="cuda")
    grid = torch.cat((grid, -grid))
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    b = scales.to(unit.dtype)
    sc = torch.where(b < 16, b, (16 + b % 16) * torch.exp2(torch.floor(b / 16) - 1))
    return (grid[c.int()].unflatten(-1, (-1, 16)) * (sc * unit)[..., None]).flatten(-2)


def _places(s):
    """Sequence, position, page and slot of every new token."""
    b, page = s["batch"], s["case"]["page"]
    cu = b["cu"].long()
    token = torch.arange(sum(b["new"]), device="cuda")
    seq = torch.searchsorted(cu[1:], token, right=True)
    pos = b["lens"].long()[seq] - cu[seq + 1] + token
    return seq, pos, b["table"].long()[seq, pos // page], pos % page


def _append_plain(s):
    page, slot = s["slots"] // s["case"]["page"], s["slots"] % s["case"]["page"]
    unit = s["unit"][None, :, None]
    s["kc"][page, :, slot], s["ks"][page, :, slot] = _quantise4(s["k"].float(), unit)
    s["vc"][page, :, slot], s["vs"][page, :, :, slot] = _quantise4(s["v"].float(), unit)
    return s["kc"], s["vc"], s["ks"], s["vs"]


def _attn_plain(s):
    c, b = s["case"], s["batch"]
    hq, hkv, d, page, n = c["hq"], c["hkv"], c["d"], c["page"], max(b["new"])
    seqs, width = b["table"].shape
    seq, pos, _, _ = _places(s)
    row = torch.arange(seq.numel(), device="cuda") - b["cu"].long()[seq]
    q = torch.zeros((seqs, n, hq, d), device="cuda")
    q[seq, row] = s["q"].float() * s["scale"]
    q = q.view(seqs, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(seqs, hkv, -1, d)

    def pages(codes, scales):  # [seqs, hkv, tokens, d]
        x = _values4(codes[b["table"].long()], scales[b["table"].long()], s["unit"][:, None, None])
        return x.permute(0, 2, 1, 3, 4).reshape(seqs, hkv, width * page, d)

    scores = torch.matmul(q, pages(s["kc"], s["ks"]).transpose(2, 3).contiguous())
    key = torch.arange(width * page, device="cuda")[None, None, :]
    at = (b["lens"].long() - b["cu"].long().diff())[:, None] + torch.arange(n, device="cuda")
    at = at[:, :, None]
    see = key < b["lens"][:, None, None]
    if c["causal"]:
        see = see & (key <= at)
        if c["window"]:
            see = see & (key > at - c["window"])
    see = see.expand(seqs, n, -1)[:, None, None]
    scores = scores.view(seqs, hkv, hq // hkv, n, -1).masked_fill_(~see, float("-inf"))
    scores -= scores.amax(-1, keepdim=True).clamp(min=-1e38)
    p = scores.exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs, hkv, -1, width * page), pages(s["vc"], s["vs"].transpose(2, 3)))
    o = o.view(seqs, hkv, hq // hkv, n, d) / torch.where(total > 0, total, 1)
    return o.permute(0, 3, 1, 2, 4).reshape(seqs, n, hq, d)[seq, row].to(s["q"].dtype)


def _run_own(s):
    from w4a8_codebook_gemm_amd import serving as S
    c = s["case"]
    if c["op"] == "norm":
        p = S.add_norm_prepare(s["x"], s["w"], s["r"], eps=EPS, weight_offset=1.0,
                               normed_dtype=_type(c["y"]) if c["y"] else None)
        return p.h, p.x_q, p.s_x, p.normed
    if c["op"] == "assign":
        b = S.pages_assign(s["pages"], s["new"], s["tokens"], out=s["batch"])
        return dict(table=s["table"], cu=b.cu_tokens, lens=b.seq_lens, positions=b.positions, slots=b.slots,
                    count=b.free_count, missing=b.missing)
    if c["op"] == "release":
        lens, count = S.pages_release(s["pages"], s["keep"], in_place=False)
        return dict(stack=s["stack"], lens=lens, count=count)
    if c["op"] == "append":
        S.kv4_append(s["k"], s["v"], s["cache"], s["slots"])
        return s["kc"], s["vc"], s["ks"], s["vs"]
    return S.kv4_attention(s["q"], s["cache"], s["seqs"], scale=s["scale"], causal=c["causal"],
                           window=c["window"] if c["causal"] else 0, workspace=s["workspace"])


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "assign": _assign_plain, "release": _release_plain, "append": _append_plain,
            "attn": _attn_plain}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------- from the definitions, in 64 bits

def _norm_exact(s):
    c = s["case"]
    h = (s["x"].float() + s["r"].float()).to(s["r"].dtype).double()
    y = h / (h.pow(2).sum(-1, keepdim=True) / c["k"] + EPS).sqrt() * (1.0 + s["w"].double())
    i = torch.arange(256, device="cuda")
    bits = (i[:, None] & i[None, :])[..., None] >> torch.arange(8, device="cuda") & 1
    hadamard = 1.0 - 2.0 * (bits.sum(-1) % 2).double()
    z = (y.view(-1, 256) @ hadamard / 16).view_as(y)
    scale = z.abs().max(-1).values / 127
    return h, torch.round(z / scale[:, None]).to(torch.int8), scale, y if c["y"] else None


def _assign_exact(s):
    page, c = s["case"]["page"], s["case"]
    new, lens = _lengths(c)
    table, stack = s["table"].cpu().clone(), s["stack"].tolist()
    count, cu, missing = int(s["count"]), [0], 0
    positions, slots = [], []
    for b, (n, length) in enumerate(zip(new, lens)):
        for entry in range(-(-(length - n) // page), -(-length // page)):
            if count > 0:
                count -= 1
                table[b, entry] = stack[count]
            else:
                table[b, entry] = -1
                missing += 1
        row = table[b].tolist()
        positions += range(length - n, length)
        slots += [row[p // page] * page + p % page if row[p // page] >= 0 else -1 for p in range(length - n, length)]
        cu.append(cu[-1] + n)
    pad = s["tokens"] - len(slots)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(table=table.cuda(), cu=i32(cu), lens=i32(lens), positions=i32(positions + [0] * pad),
                slots=torch.tensor(slots + [-1] * pad, device="cuda"), count=i32([count]), missing=i32([missing]))


def _release_exact(s):
    page = s["case"]["page"]
    stack, count, table = s["stack"].tolist(), int(s["count"]), s["table"].tolist()
    keep, lens = s["keep"].tolist(), s["lens"].tolist()
    for b in reversed(range(len(lens))):
        for entry in reversed(range(-(-keep[b] // page), -(-lens[b] // page))):
            stack[count] = table[b][entry]
            count += 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(stack=i32(stack), lens=i32(keep), count=i32([count]))


def _append_exact(s):
    page, c = s["case"]["page"], s["case"]
    hkv, d = c["hkv"], c["d"]
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    steps = torch.tensor([b if b < 16 else (16 + b % 16) * 2 ** (b // 16 - 1) for b in range(256)], dtype=torch.float64, device="cuda")

    def nearest(x, points):  # ties to the even index
        hi = torch.searchsorted(points, x.contiguous()).clamp(1, len(points) - 1)
        up, down = points[hi] - x, x - points[hi - 1]
        return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)

    out = []
    for x in (s["k"], s["v"]):
        x = x.double().reshape(-1, hkv, d // 16, 16)
        byte = nearest(x.abs().max(-1).values / (6 * UNIT), steps).clamp(min=1)
        code = nearest((x / (steps[byte] * UNIT)[..., None]).abs(), grid) + 8 * torch.signbit(x)
        code = code.reshape(-1, hkv, d // 2, 2)
        out.append(((code[..., 0] + 16 * code[..., 1]).to(torch.uint8), byte.to(torch.uint8)))
    kc, vc, ks, vs = (s[n].clone() for n in ("kc", "vc", "ks", "vs"))
    for i, at in enumerate(s["slots"].tolist()):
        p, slot = divmod(at, page)
        kc[p, :, slot], ks[p, :, slot] = out[0][0][i], out[0][1][i]
        vc[p, :, slot], vs[p, :, :, slot] = out[1][0][i], out[1][1][i]
    return kc, vc, ks, vs


def _attn_exact(s):
    c, b = s["case"], s["batch"]
    group, page = c["hq"] // c["hkv"], c["page"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    unit = torch.tensor(UNIT, dtype=torch.float64, device="cuda")
    at = 0
    for j, (n, length) in enumerate(zip(b["new"], b["lengths"])):
        table = b["table"][j, :-(-length // page)].long()
        place = torch.arange(length - n, length, device="cuda")[:, None]
        key = torch.arange(length, device="cuda")[None, :]
        hide = torch.zeros((n, length), dtype=torch.bool, device="cuda")
        if c["causal"]:
            hide = key > place
            if c["window"]:
                hide |= place - key >= c["window"]
        for h in range(c["hkv"]):
            k = _values4(s["kc"][table, h], s["ks"][table, h], unit).flatten(0, 1)[:length]
            v = _values4(s["vc"][table, h], s["vs"][table, h].transpose(1, 2), unit).flatten(0, 1)[:length]
            for g in range(group):
                z = (s["q"][at:at + n, h * group + g].double() @ k.t()) * s["scale"]
                z[hide] = float("-inf")
                out[at:at + n, h * group + g] = torch.softmax(z, -1) @ v
        at += n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _norm_exact, "assign": _assign_exact, "release": _release_exact, "append": _append_exact,
            "attn": _attn_exact}[case["op"]](s)
