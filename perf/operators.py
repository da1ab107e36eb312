"""Timing cases of the attention operators: head norm + rotary positions, the int8 paged
cache's append, and attention over that cache.

Every case is one pass of one operator.  Where `own` is false `run` computes it with
elementary torch operations in 32 bits (angles in 64); where it is true it calls the
package's kernels.  `exact` computes the same from the definitions in 64 bits.

Definitions (all arithmetic below in the stated width, one rounding to the output type):

  qk_norm_rope   y = x * rsqrt(mean(x^2) + eps) * (w + offset) over a head's D values; then the
                 first R of them rotate in pairs by angle pos * inv_freq[i], cos and sin times
                 attn_factor; pairs are (i, i + R/2) or (2i, 2i + 1)
  kv_append      a page holds P tokens of one head as int8 codes with one fp32 scale.  The page
                 of a new token at slot 0 is fresh: s = max|x| / 127 over the tokens it gets.
                 Otherwise s grows by the smallest power of two 2^k, k >= 0, with
                 max|x_new| <= fl32(127 s) 2^k, and the codes before the new ones become
                 rint(c 2^-k) (a page of scale 0 takes max|x_new| / 127).
                 c = clamp(rint(fl32(x / s)), -127, 127), 0 where s = 0
  kv_attention   token i of the n new ones of a sequence of length len (new ones included) sits
                 at position p = len - n + i and sees positions max(0, p - window + 1) .. p (all
                 of 0 .. len - 1 where the case is not causal); softmax(scale q.k) v over them,
                 k and v being code times page scale
"""
import math
import random

import torch

own = False

EPS = 1e-6


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one generated token of the hybrid decoder's attention layers (24 / 4 heads of 256, a
        # quarter of the head rotated, the query projection carries a gate beside each head),
        # 200,000 tokens into its context: latency
        dict(name="rope 1 token", op="rope", tokens=1, hq=24, hkv=4, d=256, rotary=64, interleaved=False, gated=True,
             yarn=False, dtype="bf16", out="bf16", far=200000),
        # a ragged prompt in fp32, whole heads of 128 in interleaved pairs, a context stretched
        # eightfold
        dict(name="rope 1021 fp32 stretched", op="rope", tokens=1021, hq=32, hkv=8, d=128, rotary=128, interleaved=True,
             gated=False, yarn=True, dtype="f32", out="f32", far=100000),
        # a long prompt's projections, fp32 as the quantised product gives them by default, to bf16
        dict(name="rope 8192 tokens", op="rope", tokens=8192, hq=24, hkv=4, d=256, rotary=64, interleaved=False, gated=True,
             yarn=False, dtype="f32", out="bf16", far=0),
        # one new token for each of 61 sequences: most land inside a page that is partly filled
        dict(name="append 61 x 1", op="append", seqs=61, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=4000, hkv=4, d=256, page=64,
             dtype="bf16", ragged=11),
        # three prompts, of which the later chunks continue partly filled pages
        dict(name="append 3 x 2731", op="append", seqs=3, new_lo=2731, new_hi=2731, ctx_lo=0, ctx_hi=500, hkv=4, d=256,
             page=64, dtype="bf16", ragged=12),
        # decode of one short conversation: latency
        dict(name="decode 1 x 777", op="attn", seqs=1, new_lo=1, new_hi=1, ctx_lo=776, ctx_hi=776, hq=24, hkv=4, d=256,
             page=16, window=0, causal=True, dtype="bf16", ragged=21),
        # decode of a served batch of ragged lengths
        dict(name="decode 32 ragged", op="attn", seqs=32, new_lo=1, new_hi=1, ctx_lo=300, ctx_hi=16000, hq=24, hkv=4, d=256,
             page=64, window=0, causal=True, dtype="bf16", ragged=22),
        # decode far into the model's context of 262,144 tokens
        dict(name="decode 4 long", op="attn", seqs=4, new_lo=1, new_hi=1, ctx_lo=90001, ctx_hi=131072, hq=24, hkv=4, d=256,
             page=128, window=0, causal=True, dtype="bf16", ragged=23),
        # draft tokens verified together, fp32 activations, heads of 128
        dict(name="verify 16 x 4 fp32", op="attn", seqs=16, new_lo=2, new_hi=5, ctx_lo=200, ctx_hi=4096, hq=32, hkv=8, d=128,
             page=32, window=0, causal=True, dtype="f32", ragged=24),
        # chunks of two prompts that already have a context
        dict(name="prefill 2 x 2048 + 14k", op="attn", seqs=2, new_lo=1900, new_hi=2048, ctx_lo=14000, ctx_hi=14500, hq=24,
             hkv=4, d=256, page=64, window=0, causal=True, dtype="bf16", ragged=25),
        # fresh ragged prompts, heads of 128
        dict(name="prefill 5 ragged", op="attn", seqs=5, new_lo=150, new_hi=4000, ctx_lo=0, ctx_hi=0, hq=32, hkv=8, d=128,
             page=32, window=0, causal=True, dtype="bf16", ragged=26),
        # a sliding window, one cache head for each query head, heads of 64, fp32, chunks of odd sizes
        dict(name="window 7 ragged fp32", op="attn", seqs=7, new_lo=1, new_hi=700, ctx_lo=0, ctx_hi=2000, hq=16, hkv=16, d=64,
             page=16, window=512, causal=True, dtype="f32", ragged=27),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 5, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 6, 7, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128])
    op = rng.choice(["rope", "append", "attn", "attn", "attn"])
    ragged = rng.randrange(1 << 30)
    if op == "rope":
        return dict(op="rope", tokens=_log_int(rng, 1, 8192 * 4096 // max(4096, (hq + hkv) * d)), hq=hq, hkv=hkv, d=d,
                    rotary=16 * rng.randint(1, d // 16), interleaved=rng.random() < 0.5, gated=rng.random() < 0.5,
                    yarn=rng.random() < 0.5, dtype=dtype, out=rng.choice(["bf16", dtype]), far=_log_int(rng, 1, 262144))
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
    return 2 if name == "bf16" else 4


def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "rope":
        heads = case["tokens"] * (case["hq"] + hkv)
        return {"bytes": heads * d * (_size(case["dtype"]) + _size(case["out"])) + 4 * case["tokens"] + 8 * d,
                "flops": heads * (5 * d + 3 * case["rotary"])}
    new, lens = _lengths(case)
    if case["op"] == "append":
        values = 2 * sum(new) * hkv * d
        return {"bytes": values * (_size(case["dtype"]) + 1) + 8 * case["seqs"], "flops": 4 * values}
    pairs, tokens = _seen(case)
    scales = 2 * 4 * hkv * (tokens // case["page"] + case["seqs"])
    return {"bytes": 2 * sum(new) * case["hq"] * d * _size(case["dtype"]) + 2 * tokens * hkv * d + scales,
            "flops": 4 * pairs * case["hq"] * d}


# ----------------------------------------------------------------------------- inputs

def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _frequencies(case):
    """inv_freq (fp64) of base 1e7, and for a stretched context the ramp between the plain
    and the eight times slower frequencies with its factor on cos and sin."""
    r, base = case["rotary"], 1e7
    f = torch.tensor([base ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64, device="cuda")
    if not case["yarn"]:
        return f, 1.0
    edge = [r * math.log(32768 / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
    low, high = max(0, math.floor(edge[0])), min(r - 1, math.ceil(edge[1]))
    ramp = ((torch.arange(r // 2, dtype=torch.float64, device="cuda") - low) / max(high - low, 1e-3)).clamp(0, 1)
    return f / 8 * ramp + f * (1 - ramp), 0.1 * math.log(8.0) + 1.0


def _batch(case, gen):
    """Page table (pages in random order), offsets of the new tokens, lengths."""
    new, lens = _lengths(case)
    page = case["page"]
    width = max(-(-length // page) for length in lens)
    counts = torch.tensor([-(-length // page) for length in lens], device="cuda")
    pages = int(sum(-(-length // page) for length in lens))
    order = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    table = torch.zeros((case["seqs"], width), dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None, :] < counts[:, None]] = order
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    return dict(table=table, cu=torch.tensor(off, dtype=torch.int32, device="cuda"),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), pages=pages, new=new, lengths=lens)


def _filled_cache(case, pages, gen, spread):
    """Codes and scales of pages of keys or values: normal values, some channels wide, the
    scale of a page its largest magnitude over 127."""
    hkv, page, d = case["hkv"], case["page"], case["d"]
    wide = 1.0 + 3.0 * (torch.rand((1, hkv, 1, d), generator=gen, device="cuda") > 0.95)
    codes = torch.empty((pages, hkv, page, d), dtype=torch.int8, device="cuda")
    scales = torch.empty((pages, hkv), device="cuda")
    step = max(1, (1 << 26) // (hkv * page * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn((n, hkv, page, d), generator=gen, device="cuda") * wide
        x *= spread * torch.exp(0.3 * torch.randn((n, hkv, 1, 1), generator=gen, device="cuda"))
        s = x.abs().amax((2, 3)) / 127
        scales[p:p + n] = s
        codes[p:p + n] = torch.round(x / s[:, :, None, None]).clamp(-127, 127).to(torch.int8)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    d, hkv = case["d"], case["hkv"]
    state = dict(case=case)
    if case["op"] == "rope":
        m, hq, dt = case["tokens"], case["hq"], _type(case["dtype"])
        # the query projection as it comes: [head, query | gate] where there is a gate
        q = (rand(m, hq, 2 * d if case["gated"] else d) * 2).to(dt)
        state |= dict(q=q[:, :, :d], k=(rand(m, hkv, d) * 2).to(dt),
                      positions=(torch.arange(m, device="cuda") + case["far"]).to(torch.int32),
                      qw=rand(d) * 0.2, kw=rand(d) * 0.2)
        state["inv_freq"], state["factor"] = _frequencies(case)
        return state
    b = _batch(case, gen)
    m = sum(b["new"])
    state |= dict(batch=b)
    kc, ks = _filled_cache(case, b["pages"], gen, 1.0)
    vc, vs = _filled_cache(case, b["pages"], gen, 0.5)
    state |= dict(kc=kc, ks=ks, vc=vc, vs=vs)
    if case["op"] == "append":
        # keys from the norm and rotation, values as a part of a projection's wider rows
        state |= dict(k=(rand(m, hkv, d) * 1.2).to(_type(case["dtype"])),
                      v=(rand(m, 2 * hkv, d) * 0.6).to(_type(case["dtype"]))[:, hkv:])
    else:
        state |= dict(q=rand(m, case["hq"], d).to(_type(case["dtype"])), scale=d ** -0.5)
    if own:
        from w4a8_codebook_gemm_amd import attention as A
        state["cache"] = A.KVCache(kc, vc, ks, vs)
        state["seqs"] = A.Sequences(b["table"], b["cu"], b["lens"])
        if case["op"] == "attn":
            state["workspace"] = A.kv_attention_workspace(m, case["seqs"], case["hq"], hkv, d, device="cuda")
    return state


# ----------------------------------------------------------------------------- the plain forms

def _rope_plain(s):
    c = s["case"]
    half, r = c["rotary"] // 2, c["rotary"]
    angle = s["positions"].double()[:, None] * s["inv_freq"][None, :]
    cos = (angle.cos() * s["factor"]).float()[:, None, :]
    sin = (angle.sin() * s["factor"]).float()[:, None, :]

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (w + 1.0)
        y = x.clone()
        if c["interleaved"]:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            y[..., 0:r:2] = a * cos - b * sin
            y[..., 1:r:2] = b * cos + a * sin
        else:
            a, b = x[..., :half], x[..., half:r]
            y[..., :half] = a * cos - b * sin
            y[..., half:r] = b * cos + a * sin
        return y.to(_type(c["out"]))

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _places(s):
    """Sequence, position, page and slot of every new token."""
    b, page = s["batch"], s["case"]["page"]
    cu = b["cu"].long()
    token = torch.arange(sum(b["new"]), device="cuda")
    seq = torch.searchsorted(cu[1:], token, right=True)
    pos = b["lens"].long()[seq] - cu[seq + 1] + token
    return seq, pos, b["table"].long()[seq, pos // page], pos % page


def _append_plain(s):
    page, b = s["case"]["page"], s["batch"]
    _, _, pages, slot = _places(s)
    first = torch.full((b["pages"],), page, device="cuda").scatter_reduce(0, pages, slot, "amin")
    touched = (first < page)[:, None]
    fresh = (first == 0)[:, None]
    c127 = torch.tensor(127.0, device="cuda")
    # only a sequence's first page can hold codes from before
    lead = b["table"].long().gather(1, ((b["lens"] - b["cu"].diff()) // page).long()[:, None])[:, 0]
    before = torch.arange(page, device="cuda")[None, None, :, None] < first[lead][:, None, None, None]

    def one(x, codes, scales):
        x = x.float()
        amax = torch.zeros_like(scales).scatter_reduce(0, pages[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        ma, ea = torch.frexp(amax)
        ms, es = torch.frexp(scales * c127)
        grow = torch.where((amax > 0) & (scales > 0), (ea - es + (ma > ms).int()).clamp(min=0), 0)
        grown = scales * torch.exp2((grow // 2).float()) * torch.exp2((grow - grow // 2).float())
        new = torch.where(fresh | (scales == 0), amax / c127, grown)
        new = torch.where(touched, new, scales)
        shift = torch.exp2(-(grow * (touched & ~fresh)).clamp(max=60).float())[lead][:, :, None, None]
        old = codes[lead]
        codes[lead] = torch.where(before, torch.round(old.float() * shift).to(torch.int8), old)
        st = new[pages][:, :, None]
        q = torch.where(st > 0, torch.round(x / st), 0).clamp(-127, 127)
        codes[pages, :, slot] = q.to(torch.int8)
        scales.copy_(new)

    one(s["k"], s["kc"], s["ks"])
    one(s["v"], s["vc"], s["vs"])
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
        x = codes[b["table"].long()].float() * scales[b["table"].long()][..., None, None]
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
    o = torch.matmul(p.view(seqs, hkv, -1, width * page), pages(s["vc"], s["vs"]))
    o = o.view(seqs, hkv, hq // hkv, n, d) / torch.where(total > 0, total, 1)
    return o.permute(0, 3, 1, 2, 4).reshape(seqs, n, hq, d)[seq, row].to(s["q"].dtype)


def _run_own(s):
    from w4a8_codebook_gemm_amd import attention as A
    c = s["case"]
    if c["op"] == "rope":
        return A.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                              weight_offset=1.0, interleaved=c["interleaved"], attn_factor=s["factor"],
                              out_dtype=_type(c["out"]))
    if c["op"] == "append":
        A.kv_append(s["k"], s["v"], s["cache"], s["seqs"])
        return s["kc"], s["vc"], s["ks"], s["vs"]
    return A.kv_attention(s["q"], s["cache"], s["seqs"], scale=s["scale"], causal=c["causal"],
                          window=c["window"] if c["causal"] else 0, workspace=s["workspace"])


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _rope_plain, "append": _append_plain, "attn": _attn_plain}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------- from the definitions, in 64 bits

def _rope_exact(s):
    c = s["case"]
    r = c["rotary"]
    i = torch.arange(r // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
    turn = torch.polar(torch.full((c["tokens"], r // 2), float(s["factor"]), dtype=torch.float64, device="cuda"),
                       torch.outer(s["positions"].double(), s["inv_freq"]))
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.double()
        x = x / ((x * x).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * (1.0 + w.double())
        z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        x[..., first], x[..., second] = z.real, z.imag
        out.append(x)
    return tuple(out)


def _append_exact(s):
    c, b = s["case"], s["batch"]
    out = []
    for x, codes, scales in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        codes, scales = codes.clone(), scales.double()
        at = 0
        for j, (n, length) in enumerate(zip(b["new"], b["lengths"])):
            table = b["table"][j].tolist()
            pos = length - n
            while pos < length:
                page, slot = table[pos // c["page"]], pos % c["page"]
                take = min(length - pos, c["page"] - slot)
                y = x[at:at + take].double().transpose(0, 1)          # [hkv, take, d]
                top = y.abs().amax((1, 2))
                old = scales[page].clone()
                # 127 times the scale is held in 32 bits, as the scale is
                room = (old.float().double() * 127).float().double()
                k = torch.ceil(torch.log2(top / room)).nan_to_num(0, 0, 0)
                k = torch.where(room * torch.exp2(k - 1) >= top, k - 1, k)
                k = torch.where(room * torch.exp2(k) < top, k + 1, k).clamp(min=0)
                start = torch.full_like(old, slot == 0, dtype=torch.bool) | (old == 0)
                new = torch.where(start, top / 127, old * torch.exp2(k))
                k = torch.where(start, 0, k)
                codes[page, :, :slot] = torch.round(codes[page, :, :slot].double() * torch.exp2(-k)[:, None, None]).to(torch.int8)
                held = new.float().double()[:, None, None]
                code = torch.where(held > 0, torch.round((y / held).float()), 0).clamp(-127, 127)
                codes[page, :, slot:slot + take] = code.to(torch.int8)
                scales[page] = new
                pos, at = pos + take, at + take
        out.append((codes, scales))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _attn_exact(s):
    c, b = s["case"], s["batch"]
    group, page = c["hq"] // c["hkv"], c["page"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
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
            k = (s["kc"][table, h].double() * s["ks"][table, h, None, None].double()).flatten(0, 1)[:length]
            v = (s["vc"][table, h].double() * s["vs"][table, h, None, None].double()).flatten(0, 1)[:length]
            for g in range(group):
                z = (s["q"][at:at + n, h * group + g].double() @ k.t()) * s["scale"]
                z[hide] = float("-inf")
                out[at:at + n, h * group + g] = torch.softmax(z, -1) @ v
        at += n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _rope_exact, "append": _append_exact, "attn": _attn_exact}[case["op"]](s)
