"""Performance cases of the softmax-attention layers of a hybrid stack in serving: rotary
positions, and a paged cache held in 8 bits.

Four operators, each in a plain form (elementary torch operations in fp32, angles in 64
bits) and, where ``own`` is set, through the framework's public calls:

  rotary     the pairs of a part of each head turned by position * inv_freq[j], of q and k,
             forward or backward (the gradients turned the other way)
  plan       from the requests' lengths: blocks taken from a free list into the block table
             (those of ended requests returned first), row starts, positions, and the slot of
             each new token
  write      new keys and values rounded to e4m3 into the slots, with one scale for each block
             of tokens and head; a block that grows keeps the larger scale of its parts
  attention  softmax(scale q k^T) v of each request's new tokens over its cached ones, its own
             among them (causal), heads in groups that share a key and value head

A case is a dict of plain values.  The lengths of a batch are part of the case: listed in
``past`` and ``new``, or drawn from ``lo`` to ``hi`` by the number ``mix``.  A scale is the
smallest power of two (2^-60 at least) under which the largest value is at most 448.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_E4M3 = torch.float8_e4m3fn
_SPARE = 8      # blocks of the pool beyond those that a case needs


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _ints(text):
    return [int(x) for x in str(text).split(",")]


def _up(a, b):
    return -(-a // b)


def _lens(case):
    """(past, new) of each request, two lists of whole numbers."""
    if "past" in case:
        return _ints(case["past"]), _ints(case["new"])
    rng = random.Random(case["mix"])
    return [rng.randint(case["lo"], case["hi"]) for _ in range(case["N"])], [1] * case["N"]


# ---------------------------------------------------------------- the cases
def _rotary(name, T, Hq, Hk, d, rot, first, inter, dtype, far, scaled, backward):
    return dict(name=name, op="rotary", T=T, Hq=Hq, Hk=Hk, d=d, rot=rot, first=first, inter=inter,
                dtype=dtype, far=far, scaled=scaled, backward=backward)


_RAGGED = "12837,1520,9301,16001,655,4099,7777,2048,14530,3001,511,10240,6213,12000,901,8190"
_SIXTEEN_NONE = ",".join(["0"] * 16)


def listed():
    return [
        # the token of one request far into a long context: latency
        _rotary("rotary_token", 1, 32, 8, 128, 128, 0, False, "bf16", True, "yarn", False),
        # the long prompt, 96 query heads, the last 64 channels of each head turned
        _rotary("rotary_64k", 65536, 96, 8, 128, 64, 64, True, "bf16", False, "none", False),
        # the backward of a 4K training sequence in fp32, an odd row count and head count
        _rotary("rotary_backward_f32", 4099, 9, 3, 64, 64, 0, False, "f32", False, "linear", True),
        # a decode step's bookkeeping: 256 requests, one new token each
        dict(name="plan_decode", op="plan", N=256, lo=512, hi=16384, mix=1, block=64, rows=256,
             ended=0),
        # 16 ragged prompts admitted at once in a padded batch, two requests ended before them
        dict(name="plan_prompts", op="plan", past=_SIXTEEN_NONE + ",5000,777",
             new=_RAGGED + ",-1,-1", block=16, rows=114688, ended=2),
        # a decode step's keys and values: one token for each of 256 requests
        dict(name="write_decode", op="write", N=256, lo=512, hi=4096, mix=2, block=64, Hkv=8,
             d=128, dtype="bf16"),
        # the long prompt's keys and values
        dict(name="write_64k", op="write", past="0", new="65536", block=64, Hkv=8, d=128,
             dtype="bf16"),
        # ragged prompts behind cached tokens, in fp32, small blocks, three heads
        dict(name="write_ragged_f32", op="write", past="5,0,129,64,1000", new="1000,37,2049,1,515",
             block=16, Hkv=3, d=64, dtype="f32"),
        # one request being answered: 8K cached tokens, latency
        dict(name="attention_b1", op="attention", past="8191", new="1", block=64, Hq=32, Hkv=8,
             d=128, dtype="bf16"),
        # a decode batch of 128 ragged requests: 1.1 M cached tokens, 2.2 GB
        dict(name="attention_b128", op="attention", N=128, lo=512, hi=16384, mix=3, block=64,
             Hq=32, Hkv=8, d=128, dtype="bf16"),
        # a 4K piece of a prompt behind 12K cached tokens
        dict(name="attention_prompt", op="attention", past="12288", new="4096", block=64, Hq=32,
             Hkv=8, d=128, dtype="bf16"),
        # prompts, single tokens and an idle request in one batch, fp32, odd head counts
        dict(name="attention_mixed_f32", op="attention", past="5,2000,129,64,1000,0",
             new="300,1,7,0,1,515", block=16, Hq=15, Hkv=3, d=64, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _pieces(rng, total, n):
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def draw(rng):
    op = rng.choice(["rotary", "rotary", "plan", "write", "attention", "attention", "attention"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([32, 64, 128, 128])
    block = rng.choice([16, 32, 64, 128])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    if op == "rotary":
        Hq, Hk = _log(rng, 1, 96), rng.randint(0, 8)
        most = 300_000_000 // (d * (Hq + Hk))
        rot = 16 * rng.randint(1, d // 16)
        c = _rotary("", min(_log(rng, 1, 65536), most), Hq, Hk, d, rot,
                    8 * rng.randint(0, (d - rot) // 8), rng.random() < 0.5, dtype,
                    rng.random() < 0.4, rng.choice(["none", "linear", "yarn"]), rng.random() < 0.4)
    elif op == "plan":
        if rng.random() < 0.5:
            N = _log(rng, 1, 1024)
            lo = rng.randint(0, 2000)
            c = dict(op=op, N=N, lo=lo, hi=lo + _log(rng, 1, 16000), mix=rng.randrange(1 << 30),
                     block=block, rows=N + rng.randint(0, 40), ended=0)
        else:
            N, total, ended = _log(rng, 1, 64), _log(rng, 64, 100_000), rng.randint(0, 4)
            past = [rng.choice([0, 0, rng.randint(0, 5000)]) for _ in range(N + ended)]
            new = _pieces(rng, total, N) + [-1] * ended
            c = dict(op=op, past=",".join(map(str, past)), new=",".join(map(str, new)),
                     block=block, rows=total + rng.randint(0, 1000), ended=ended)
    else:
        Hkv = rng.randint(1, 12)
        kind = rng.random()
        if kind < 0.5:      # one token for each request
            most = (1 << 29) // (Hkv * d)
            N = _log(rng, 1, 256)
            lo = rng.randint(0, 600)
            c = dict(op=op, N=N, lo=lo, hi=lo + max(1, min(_log(rng, 16, 60_000), most // N - lo)),
                     mix=rng.randrange(1 << 30))
        else:               # prompts, some of them behind cached tokens
            N = _log(rng, 1, 12)
            # for attention at most 2e9 scores, in batches padded to the longest of each
            most = 30_000 if op == "write" else min(4000, math.isqrt(10 ** 9 // (N * group * Hkv)))
            total = _log(rng, 4, max(5, most))
            reach = max(1, min(8000, 10 ** 9 // (N * total * group * Hkv)))
            past = [rng.choice([0, rng.randint(0, reach)]) for _ in range(N)]
            c = dict(op=op, past=",".join(map(str, past)),
                     new=",".join(map(str, _pieces(rng, total, N))))
        c.update(block=block, Hkv=Hkv, d=d, dtype=dtype)
        if op == "attention":
            c.update(Hq=Hkv * group)
    c.pop("name", None)
    return c


# ------------------------------------------------------------------- inputs
def _frequencies(rot, scaled):
    """inv_freq [rot / 2] in 64 bits and the factor on the turned pairs: the geometric series of
    base 10,000 plainly, for a context eight times as long by a common factor, or by parts of the
    spectrum (the waves that fit a 4,096-token context 32 times stay, those that fit it less than
    once are stretched, between them linearly)."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaled == "linear":
        return f / 8.0, 1.0
    if scaled == "yarn":
        waves = 4096.0 * f / (2.0 * math.pi)
        keep = ((waves - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return f * keep + f / 8.0 * (1.0 - keep), 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def _pool(case, past, new):
    """Blocks that hold the requests' tokens, and the table's width, with some to spare."""
    need = [_up(p + max(n, 0), case["block"]) for p, n in zip(past, new)]
    return sum(need) + _SPARE, max(1, max(need)) + 1


def _table(past, new, case, gen, dev):
    """A block table whose rows hold the blocks of the tokens given by `past`, in no order."""
    blocks, width = _pool(case, past, new)
    order = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
    have = torch.tensor([_up(p, case["block"]) for p in past], device=dev)
    first = torch.cumsum(have, 0) - have
    col = torch.arange(width, device=dev)
    at = (first[:, None] + col[None]).clamp(max=blocks - 1)
    table = torch.where(col[None] < have[:, None], order[at], torch.zeros_like(order[at]))
    return table.contiguous(), order, int(sum(_up(p, case["block"]) for p in past)), blocks


def _cache(gen, dev, blocks, Hkv, block, d):
    """Keys or values of standard deviation 0.3 to 2.5 in e4m3, and the scales."""
    scale = torch.exp2(torch.randint(-8, -5, (blocks, Hkv), generator=gen, device=dev).float())
    x = torch.randn(blocks, Hkv, block, d, generator=gen, device=dev)
    return x.mul_(80.0).clamp_(-448.0, 448.0).to(_E4M3), scale


def _starts(lens, dev):
    cu = torch.zeros(len(lens) + 1, dtype=torch.int64)
    cu[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int64), 0)
    return cu.to(torch.int32).to(dev)


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    s = dict(case=dict(case))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if case["op"] == "rotary":
        T, dt = case["T"], _DT[case["dtype"]]
        s["q"] = normal(T, case["Hq"], case["d"]).to(dt)
        s["k"] = normal(T, case["Hk"], case["d"]).to(dt) if case["Hk"] else None
        f, s["magnitude"] = _frequencies(case["rot"], case["scaled"])
        s["inv_freq"] = f.float().to(dev)
        if case["far"]:     # rows of many requests, anywhere in a context of 1,048,576 tokens
            s["positions"] = torch.randint(0, 1 << 20, (T,), generator=gen, device=dev,
                                           dtype=torch.int32)
        else:               # one prompt
            s["positions"] = torch.arange(T, device=dev, dtype=torch.int32)
        return s
    past, new = _lens(case)
    s["n_requests"], s["width"] = len(past), _pool(case, past, new)[1]
    if case["op"] == "plan":
        s["past"] = torch.tensor(past, dtype=torch.int32, device=dev)
        s["new"] = torch.tensor(new, dtype=torch.int32, device=dev)
        s["table"], order, used, blocks = _table(past, new, case, gen, dev)
        s["free"] = torch.full((blocks,), -1, dtype=torch.int32, device=dev)
        s["free"][:blocks - used] = order[used:]
        s["n_free"] = torch.tensor([blocks - used], dtype=torch.int32, device=dev)
        return s
    dt, Hkv, d, block = _DT[case["dtype"]], case["Hkv"], case["d"], case["block"]
    T = sum(new)
    whole = [p + n for p, n in zip(past, new)]
    s["table"], _, _, blocks = _table(whole, [0] * len(new), case, gen, dev)
    s["k_cache"], s["k_scale"] = _cache(gen, dev, blocks, Hkv, block, d)
    s["v_cache"], s["v_scale"] = _cache(gen, dev, blocks, Hkv, block, d)
    s["cu"] = _starts(new, dev)
    s["context"] = torch.tensor(whole, dtype=torch.int32, device=dev)
    n = torch.tensor(new, device=dev)
    s["request"] = torch.repeat_interleave(torch.arange(len(new), device=dev), n)
    s["index"] = torch.arange(T, device=dev) - s["cu"][s["request"]]    # within the request's rows
    if case["op"] == "write":
        s["k"], s["v"] = normal(T, Hkv, d).to(dt), normal(T, Hkv, d).to(dt)
        p = torch.tensor(past, device=dev)[s["request"]] + s["index"]
        s["slots"] = (s["table"][s["request"], p // block].long() * block + p % block).to(torch.int32)
        rows = torch.tensor([i for i, x in enumerate(new) if x > 0], device=dev)
        s["opened"] = s["slots"][s["cu"][rows].long()].long() // block  # where each request goes on
        return s
    s["q"] = normal(T, case["Hq"], d).to(dt)
    s["max_new"] = max(new)
    s["scale"] = round(d ** -0.5, 6)
    return s


# -------------------------------------------------------------- plain forms
def _turned(x, cos, sin, c):
    """The pairs of channels first .. first + rot turned; cos and sin [T, 1, rot / 2]."""
    a, b = c["first"], c["first"] + c["rot"]
    part = x[..., a:b]
    if c["inter"]:
        u, w = part[..., 0::2], part[..., 1::2]
        part = torch.stack((u * cos - w * sin, u * sin + w * cos), dim=-1).flatten(-2)
    else:
        u, w = part[..., :c["rot"] // 2], part[..., c["rot"] // 2:]
        part = torch.cat((u * cos - w * sin, u * sin + w * cos), dim=-1)
    return torch.cat((x[..., :a], part, x[..., b:]), dim=-1)


def _rotary_in(s, c, ft):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None]
    if c["backward"]:
        angle = -angle
    cos, sin = ((t * s["magnitude"]).to(ft)[:, None, :] for t in (torch.cos(angle), torch.sin(angle)))
    return {n: _turned(s[n].to(ft), cos, sin, c) for n in ("q", "k") if s[n] is not None}


def _plain_rotary(s, c):
    dt = s["q"].dtype
    return {n: x.to(dt) for n, x in _rotary_in(s, c, torch.float32).items()}


def _plain_plan(s, c):
    block, T, past, new, table, free = c["block"], c["rows"], s["past"], s["new"], s["table"], s["free"]
    W, F, dev = table.shape[1], free.shape[0], table.device
    n = new.clamp(min=0)
    end = torch.cumsum(n, 0)
    have = (past + block - 1).div(block, rounding_mode="floor")
    want = (past + n + block - 1).div(block, rounding_mode="floor")
    bad = (past < 0) | (new < -1)
    ended = (new == -1) & ~bad & (have <= W)
    wide, over = want > W, end > T
    status = torch.where(bad, 1, torch.where(wide, 2, torch.where(over, 4, 0)))
    col = torch.arange(W, device=dev)
    gone = torch.where(ended, have, 0)
    before = torch.cumsum(gone, 0) - gone
    to = s["n_free"] + before[:, None] + col[None]
    to = torch.where(ended[:, None] & (col[None] < have[:, None]) & (to < F), to, F).long()
    longer = torch.cat((free, free[:1]))
    longer.scatter_(0, to.flatten(), table.flatten())
    free.copy_(longer[:F])
    total = (s["n_free"] + gone.sum()).clamp(max=F)
    need = torch.where((status == 0) & ~ended, want - have, 0)
    upto = torch.cumsum(need, 0)
    short = (need > 0) & (upto > total)
    status = torch.where(short, 3, status)
    served = status == 0
    take = total - 1 - (upto - need)[:, None] - (col[None] - have[:, None])
    mine = (served & ~ended)[:, None] & (col[None] >= have[:, None]) & (col[None] < want[:, None])
    table.copy_(torch.where(mine, free[take.clamp(0, F - 1).long()], table))
    left = total - torch.where(served, need, 0).sum()
    context = torch.where(served & ~ended, past + n, 0)
    cu = torch.cat((torch.zeros_like(end[:1]), end)).clamp(max=T)
    t = torch.arange(T, device=dev)
    req = torch.searchsorted(cu[1:], t, right=True).clamp(max=len(n) - 1)
    inside = t < cu[-1]
    pos = torch.where(inside, past[req] + t - cu[req], 0)
    at = (pos // block).clamp(0, W - 1)
    slot = table[req, at] * block + pos % block
    slot = torch.where(inside & served[req], slot, -1)
    i32 = torch.int32
    return {"cu_seqlens": cu.to(i32), "context_lens": context.to(i32), "positions": pos.to(i32),
            "slots": slot.to(i32), "status": status.to(i32), "n_free": left.to(i32).reshape(1),
            "block_table": table, "free_blocks": free}


def _power(largest):
    """The smallest power of two, 2^-60 at least, under which `largest` is at most 448."""
    m, e = torch.frexp(largest)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-60)
    return torch.ldexp(torch.ones_like(largest), torch.where(largest > 0, e, -60))


def _written(x, cache, scale, s, block):
    """x [T, Hkv, d] into its slots; cache and scale in place."""
    T, Hkv, d = x.shape
    x = x.float()
    slots = s["slots"].long()
    blk, off = slots // block, slots % block
    largest = torch.zeros_like(scale)
    largest.scatter_reduce_(0, blk[:, None].expand(T, Hkv), x.abs().amax(dim=-1), "amax")
    first = torch.full((scale.shape[0],), block, dtype=torch.int64, device=x.device)
    first.scatter_reduce_(0, blk, off, "amin")
    fresh = _power(largest)
    grown = torch.where((first > 0)[:, None], torch.maximum(scale, fresh), fresh)
    now = torch.where((first < block)[:, None], grown, scale)
    bits = cache.view(torch.uint8)
    b = s["opened"]
    # the tokens ahead of the first new one; what lies behind stays as it is
    ahead = torch.arange(block, device=x.device)[None] < first[b][:, None]
    ratio = torch.where(ahead[:, None], (scale[b] / now[b])[..., None], 1.0)
    old = bits[b].view(_E4M3).float() * ratio[..., None]
    bits[b] = old.to(_E4M3).view(torch.uint8)
    rounded = (x / now[blk][..., None]).clamp(-448.0, 448.0).to(_E4M3)
    bits[blk, :, off] = rounded.view(torch.uint8)
    scale.copy_(now)


def _plain_write(s, c):
    _written(s["k"], s["k_cache"], s["k_scale"], s, c["block"])
    _written(s["v"], s["v_cache"], s["v_scale"], s, c["block"])
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _attended(s, c, ft, heads=None):
    """o [T, Hq, d] of the given key and value heads (all without), in the type ft."""
    heads = slice(None) if heads is None else heads
    table, block = s["table"].long(), c["block"]
    N, W = table.shape
    G, L, n_max = c["Hq"] // c["Hkv"], W * block, s["max_new"]

    def rows(cache, scale):
        x = cache.view(torch.uint8)[:, heads][table].view(_E4M3).to(ft)     # [N, W, Hkv, block, d]
        x = x * scale[:, heads][table].to(ft)[..., None, None]
        return x.transpose(1, 2).reshape(N, -1, L, c["d"])

    dev, ctx = table.device, s["context"].long()
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    key, j = torch.arange(L, device=dev), torch.arange(n_max, device=dev)
    K = rows(s["k_cache"], s["k_scale"])
    V = torch.where((key[None] < ctx[:, None])[:, None, :, None], rows(s["v_cache"], s["v_scale"]), 0.0)
    T, H = s["q"].shape[0], K.shape[1]
    at = (s["cu"][:-1, None].long() + j[None]).clamp(max=T - 1)
    q = s["q"].view(T, c["Hkv"], G, c["d"])[:, heads][at].to(ft)            # [N, n_max, Hkv, G, d]
    q = q.permute(0, 2, 3, 1, 4).reshape(N, H, G * n_max, c["d"])
    last = (ctx - n)[:, None] + j[None]                                     # the last key of a row
    seen = (key[None, None] <= last[:, :, None]) & (j[None] < n[:, None])[:, :, None]
    x = torch.matmul(q, K.transpose(2, 3)).mul_(s["scale"]).view(N, H, G, n_max, L)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    x.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = x.sum(dim=-1, keepdim=True)
    o = torch.matmul(x.view(N, H, G * n_max, L), V).view(N, H, G, n_max, c["d"])
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4)       # [N, n_max, Hkv, G, d]
    return o[s["request"], s["index"]].reshape(T, H * G, c["d"])


def _plain_attention(s, c):
    return {"o": _attended(s, c, torch.float32).to(s["q"].dtype)}


_PLAIN = dict(rotary=_plain_rotary, plan=_plain_plan, write=_plain_write,
              attention=_plain_attention)


# ----------------------------------------------------------- framework calls
def _own_run(s, c):
    import kimi_delta_attention_12_gb300 as kda
    if c["op"] == "rotary":
        call = kda.kda_rotary_backward if c["backward"] else kda.kda_rotary
        q, k = call(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=c["inter"],
                    first=c["first"], magnitude=s["magnitude"])
        return {"q": q} if k is None else {"q": q, "k": k}
    if c["op"] == "plan":
        p = kda.kda_cache_plan(s["past"], s["new"], s["table"], s["free"], s["n_free"], c["block"],
                               c["rows"])
        return dict(p, block_table=s["table"], free_blocks=s["free"])
    if c["op"] == "write":
        kda.kda_cache_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"],
                            s["v_scale"])
        return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    return {"o": kda.kda_cache_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"],
                                         s["v_scale"], s["table"], s["context"], s["cu"],
                                         max_new=s["max_new"], scale=s["scale"])}


def run(state):
    c = state["case"]
    return _own_run(state, c) if own else _PLAIN[c["op"]](state, c)


# ------------------------------------------------------------- what it takes
def work(case):
    if case["op"] == "rotary":
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["T"] * (case["Hq"] + case["Hk"])
        return {"bytes": 2 * n * case["d"] * size + 4 * case["T"] + 2 * case["rot"],
                "flops": 3 * n * case["rot"]}
    past, new = _lens(case)
    N, T = len(new), sum(x for x in new if x > 0)
    if case["op"] == "plan":
        block = case["block"]
        held = [(_up(p, block), _up(p + n, block)) for p, n in zip(past, new) if n >= 0]
        fresh = sum(b - a for a, b in held)
        gone = sum(_up(p, block) for p, n in zip(past, new) if n < 0)
        read = sum(b - p // block for p, (a, b) in zip(past, held) if b > p // block)
        return {"bytes": 4 * (2 * N + 3 * N + 3 + 2 * case["rows"] + 2 * fresh + read + 2 * gone),
                "flops": 0}
    size, Hkv, d = (2 if case["dtype"] == "bf16" else 4), case["Hkv"], case["d"]
    if case["op"] == "write":
        runs = sum(_up(p + n, case["block"]) - p // case["block"] for p, n in zip(past, new) if n)
        return {"bytes": T * (2 * Hkv * d * (size + 1) + 4) + 16 * runs * Hkv,
                "flops": 4 * T * Hkv * d}
    ctx = [p + n for p, n in zip(past, new)]
    blocks = sum(_up(x, case["block"]) for x, n in zip(ctx, new) if n)
    pairs = sum(p * n + n * (n + 1) // 2 for p, n in zip(past, new))
    held = sum(x for x, n in zip(ctx, new) if n)
    return {"bytes": 2 * held * Hkv * d + blocks * (8 * Hkv + 4) + 2 * T * case["Hq"] * d * size,
            "flops": 4 * pairs * case["Hq"] * d}


# ------------------------------------------------- the definition in 64 bits
def _exact_rotary(s, c, n):
    """Each pair as a complex number times magnitude * e^{i angle}."""
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    turn = torch.polar(torch.full_like(angle, s["magnitude"]), -angle if c["backward"] else angle)
    pair = torch.arange(c["rot"] // 2, device=angle.device)
    re = c["first"] + (2 * pair if c["inter"] else pair)
    im = re + (1 if c["inter"] else c["rot"] // 2)
    x = s[n].double()
    z = torch.complex(x[..., re], x[..., im]).mul_(turn[:, None])
    x[..., re], x[..., im] = z.real, z.imag
    return x


def _exact_write(s, c, x, cache, scale):
    """(values, scales): block by block the numbers that the bytes stand for, the scale that they
    need, and the nearest of e4m3 (three bits after the leading one, exponents from -6, steps of
    2^-9 below), ties to even."""
    slots, dev = s["slots"].long(), cache.device
    blk, off = slots // c["block"], slots % c["block"]
    touched = torch.unique(blk)
    place = torch.full((scale.shape[0],), -1, dtype=torch.int64, device=dev)
    place[touched] = torch.arange(len(touched), device=dev)
    used = torch.zeros(len(touched), c["block"], dtype=torch.bool, device=dev)
    used[place[blk], off] = True
    old = torch.cumsum(used.int(), 1) == 0                  # tokens ahead of the first new one
    held = cache.view(torch.uint8)[touched].view(_E4M3).double()
    value = held * scale[touched].double()[..., None, None] * old[:, None, :, None]
    value.transpose(1, 2)[place[blk], off] = x.double()
    new = (value.abs() * used[:, None, :, None]).flatten(2).amax(-1)
    e = torch.floor(torch.log2((new / 448.0).clamp(min=2.0 ** -70)))
    e = torch.where(new <= 448.0 * torch.exp2(e), e, e + 1.0).clamp(min=-60.0)
    kept = old.any(dim=1)[:, None]
    now = torch.where(kept, torch.maximum(scale[touched].double(), torch.exp2(e)), torch.exp2(e))
    u = value / now[..., None, None]
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3.0)
    u = torch.round(u / step) * step
    values, scales = cache.double(), scale.double()
    values[touched] = torch.where((used | old)[:, None, :, None], u, held)
    scales[touched] = now
    return values, scales


def exact(case, seed):
    if case["op"] == "plan" or (case["op"] == "attention" and work(case)["flops"] > 4e12):
        return None
    s, c = prepare(case, seed), case
    if c["op"] == "rotary":
        return {n: _exact_rotary(s, c, n) for n in ("q", "k") if s[n] is not None}
    if c["op"] == "write":
        out = {}
        for n in ("k", "v"):
            out[n + "_cache"], out[n + "_scale"] = _exact_write(s, c, s[n], s[n + "_cache"],
                                                                s[n + "_scale"])
        return out
    # request by request and head by head, from the sums' definition
    T, G = s["q"].shape[0], c["Hq"] // c["Hkv"]
    o = torch.zeros(T, c["Hq"], c["d"], dtype=torch.float64, device=s["q"].device)
    starts, lens = s["cu"].tolist(), s["context"].tolist()
    for i, length in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        if a == b:
            continue
        blocks = s["table"][i, :_up(length, c["block"])].long()
        last = length - (b - a) + torch.arange(b - a, device=o.device)
        hidden = torch.arange(length, device=o.device)[None] > last[:, None]
        for h in range(c["Hkv"]):
            K, V = ((s[n + "_cache"].view(torch.uint8)[blocks, h].view(_E4M3).double()
                     * s[n + "_scale"][blocks, h].double()[:, None, None])
                    .reshape(-1, c["d"])[:length] for n in ("k", "v"))
            for g in range(h * G, (h + 1) * G):
                x = (s["q"][a:b, g].double() @ K.T) * s["scale"]
                o[a:b, g] = torch.softmax(x.masked_fill_(hidden, -math.inf), dim=-1) @ V
    return {"o": o}
