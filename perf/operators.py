"""Performance cases of the decayed linear attention and of the block norms.

Five operators, each in a plain form (elementary torch operations in fp32) and,
where ``own`` is set, through the framework's public calls:

  lin_prefill    S_t = e^{g_h} S_{t-1} + k_t v_t^T,  o_t = scale * S_t^T q_t
                 over packed sequences, with states in and out
  lin_decode     one step of the same recurrence for each of B sequences, the
                 fp32 state pool updated in place at the rows `slots`
  lin_backward   dq, dk, dv and dS0 of the prefill, given dO and dS_T
  norm           u = RMSNorm(y; w_post) * act(gate),  x' = x + res_scale * u,
                 h = RMSNorm(x'; w_pre)   (each part but the first optional)
  norm_backward  the gradients of x' and h with respect to y, gate, x and the
                 three weight vectors, the stream x' given as it was stored

A case is a dict of plain values.  Ragged batches give their lengths in
``lens``; an empty ``slots`` means the identity.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 128


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _lens(case):
    return [int(x) for x in str(case["lens"]).split(",")]


# ---------------------------------------------------------------- the cases
def _prefill(name, lens, H, dk, dv, dtype, state):
    return dict(name=name, op="lin_prefill", lens=lens, H=H, dk=dk, dv=dv, dtype=dtype,
                state=state, scale=round(dk ** -0.5, 6))


def _norm(name, op, rows, D, group, gate, residual, pre, dtype):
    return dict(name=name, op=op, rows=rows, D=D, group=group, gate=gate, residual=residual,
                pre=pre, dtype=dtype)


_RAGGED = "12837,1520,9301,16001,655,4099,7777,2048,14530,3001,511,10240,6213,12000,901,8190"


def listed():
    return [
        # the smallest workload of the inputs module: one short fp32 prompt, where launches count
        _prefill("prefill_tiny_f32", "64", 2, 32, 32, "f32", False),
        # the 4K prompt of the benchmark: few (sequence, head) pairs for the machine
        _prefill("prefill_4k", "4096", 32, 128, 128, "bf16", True),
        # a packed batch of 16 ragged prompts that continue from cached states
        _prefill("prefill_ragged", _RAGGED, 64, 128, 128, "bf16", True),
        # the benchmark's long prompt: one sequence of 65,536 tokens, 96 heads
        _prefill("prefill_64k", "65536", 96, 128, 128, "bf16", False),
        # one request being answered: latency of a single token
        dict(name="decode_b1", op="lin_decode", B=1, pool=1, H=32, dk=128, dv=128, dtype="bf16",
             slots=False, scale=round(128 ** -0.5, 6)),
        # the benchmark's decode batch: 256 requests in a pool with room, 1.6 GB of states touched
        dict(name="decode_b256", op="lin_decode", B=256, pool=300, H=96, dk=128, dv=128,
             dtype="bf16", slots=True, scale=round(128 ** -0.5, 6)),
        # a training step's backward on one 4K sequence
        dict(_prefill("backward_4k", "4096", 32, 128, 128, "bf16", False), op="lin_backward"),
        # a ragged fp32 backward with states at both ends, unequal key and value widths
        dict(_prefill("backward_ragged_f32", "1000,37,2049,1,515", 8, 64, 128, "f32", True),
             op="lin_backward"),
        # a single token's row between two blocks: latency
        _norm("norm_row", "norm", 1, 4096, 0, "sigmoid", True, True, "bf16"),
        # the per-head norm and gate after the long prompt's attention (96 heads of 128)
        _norm("norm_heads_64k", "norm", 65536, 12288, 128, "sigmoid", False, False, "bf16"),
        # the backward between two blocks of a 4K training sequence of width 4096
        _norm("norm_backward_4k", "norm_backward", 4096, 4096, 0, "sigmoid", True, True, "bf16"),
        # an odd fp32 width and row count, silu gate
        _norm("norm_backward_odd_f32", "norm_backward", 1003, 1000, 0, "silu", True, True, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _not_3072(n):
    return n + 8 if n == 3072 else n


def draw(rng):
    op = rng.choice(["lin_prefill", "lin_prefill", "lin_decode", "lin_backward", "norm",
                     "norm_backward"])
    wide = rng.random() < 0.6  # the tensor-core shape, else any of the supported ones
    dtype = "bf16" if wide or rng.random() < 0.4 else "f32"
    dk, dv = (128, 128) if wide else (rng.choice([32, 64, 128]), rng.choice([32, 64, 128]))
    scale = round(dk ** -0.5, 6)
    if op in ("lin_prefill", "lin_backward"):
        H = _log(rng, 1, 96)
        # token-head pairs, at most a tenth of the long prompt's (a fortieth for fp32)
        most = 600_000 if wide else 150_000
        total = max(1, min(_log(rng, 1, 40000), most // H))
        n = min(rng.choice([1, 1, 2, 5, 16]), total)
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        lens = ",".join(str(_not_3072(x)) for x in lens)
        c = _prefill("", lens, H, dk, dv, dtype, rng.random() < 0.5)
        c.update(op=op)
    elif op == "lin_decode":
        B = _log(rng, 1, 256)
        c = dict(op=op, B=B, pool=B + rng.randint(0, 40), H=_log(rng, 1, 96), dk=dk, dv=dv,
                 dtype=dtype, slots=rng.random() < 0.6, scale=scale)
    else:
        heads = rng.random() < 0.4
        if heads:
            group = rng.choice([32, 64, 128])
            D = group * _log(rng, 1, 96)
        else:
            group, D = 0, 8 * _log(rng, 4, 1536)
        D = D + max(group, 8) if D == 3072 else D
        rows = _not_3072(max(1, min(_log(rng, 1, 65536), 100_000_000 // D)))
        res = rng.random() < 0.7
        c = _norm("", op, rows, D, group, rng.choice(["none", "sigmoid", "silu"]), res,
                  res and rng.random() < 0.7, dtype)
    c.pop("name", None)
    return c


# ------------------------------------------------------------------- inputs
def _tensors(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = _DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def unit(*shape):
        x = normal(*shape)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    s = dict(case=dict(case))
    if case["op"].startswith("lin_"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        T = case["B"] if case["op"] == "lin_decode" else sum(_lens(case))
        # keys and queries of unit length; slopes spread over the heads as a geometric series
        s["q"], s["k"], s["v"] = unit(T, H, dk), unit(T, H, dk), normal(T, H, dv).to(dt)
        slope = torch.exp2(-8.0 * torch.arange(1, H + 1, device=dev) / H)
        s["log_decay"] = -(slope * (0.5 + torch.rand(H, generator=gen, device=dev))).float()
        if case["op"] == "lin_decode":
            s["state"] = 0.1 * normal(case["pool"], H, dk, dv)
            s["slots"] = (torch.randperm(case["pool"], generator=gen, device=dev)[:T]
                          .to(torch.int32) if case["slots"] else None)
            return s
        lens = _lens(case)
        host = torch.zeros(len(lens) + 1, dtype=torch.int32)
        host[1:] = torch.cumsum(torch.tensor(lens), 0).to(torch.int32)
        s["lens"], s["cu_host"], s["cu"] = lens, host, host.to(dev)
        s["initial_state"] = 0.1 * normal(len(lens), H, dk, dv) if case["state"] else None
        if case["op"] == "lin_backward":
            s["dO"] = normal(T, H, dv).to(dt)
            s["dS_final"] = 0.1 * normal(len(lens), H, dk, dv) if case["state"] else None
        return s
    T, D = case["rows"], case["D"]
    G = case["group"] or D
    s["y"] = (normal(T, D) * 0.5).to(dt)
    s["w_post"] = 1.0 + 0.1 * normal(G)
    s["gate"] = normal(T, D).to(dt) if case["gate"] != "none" else None
    s["x"] = normal(T, D).to(dt) if case["residual"] else None
    s["res_scale"] = 0.5 + 0.1 * normal(D) if case["residual"] else None
    s["w_pre"] = 1.0 + 0.1 * normal(D) if case["pre"] else None
    if case["op"] == "norm_backward":
        s["x_out"] = s.pop("x")   # what the stream holds after the forward
        s["dx_out"] = normal(T, D).to(dt)
        s["dh"] = normal(T, D).to(dt) if case["pre"] else None
    return s


def _chunks(lens, dev):
    """Where each chunk of up to _CHUNK tokens lies: the tables of the plain form."""
    n = torch.tensor(lens)
    per = (n + _CHUNK - 1) // _CHUNK
    seq = torch.repeat_interleave(torch.arange(len(lens)), per)
    first = torch.cumsum(per, 0) - per
    off = (torch.arange(len(seq)) - first[seq]) * _CHUNK            # within its sequence
    length = torch.minimum(n[seq] - off, torch.tensor(_CHUNK))
    bos = (torch.cumsum(n, 0) - n)[seq]
    i = torch.arange(_CHUNK)
    valid = i[None] < length[:, None]
    fwd = torch.where(valid, bos[:, None] + off[:, None] + i[None], 0)
    rev = torch.where(valid, bos[:, None] + n[seq][:, None] - 1 - off[:, None] - i[None], 0)
    return dict(lens=n.to(dev), seq=seq.to(dev), off=off.to(dev), length=length.to(dev),
                valid=valid.to(dev), fwd=fwd.to(dev), rev=rev.to(dev))


def prepare(case, seed):
    s = _tensors(case, seed)
    if "lens" in s:
        s["plan"] = _chunks(s["lens"], s["q"].device)
    return s


# --------------------------------------------------------------- plain forms
def _decayed(x, y, z, g, S_in, plan, reverse, out_scale, kv_scale):
    """out_t = out_scale * (sum over s up to t of kv_scale * e^{g(t-s)} (x_t . y_s) z_s + the
    initial state's part), over chunks; the states between the chunks by one product with the
    decays between them.  In reverse, time runs from each sequence's end and the state met by a
    token is not decayed before it."""
    idx, valid = (plan["rev"] if reverse else plan["fwd"]), plan["valid"]
    late = 1 if reverse else 0
    T, H = x.shape[:2]
    gd = g.double()
    i = torch.arange(_CHUNK, device=x.device)
    keep = valid[:, :, None, None]
    X, Y, Z = (torch.where(keep, t[idx].float(), 0.0).transpose(1, 2) for t in (x, y, z))
    dist = i[:, None] - i[None]
    W = torch.where(dist >= 0, torch.exp(gd[:, None, None] * dist.clamp(min=0)), 0.0).float()
    out = torch.matmul(torch.matmul(X, Y.transpose(2, 3)) * (W * kv_scale), Z)
    to_end = (plan["length"][:, None] - 1 - i[None] + late).clamp(min=0)
    w_end = torch.exp(gd[None, :, None] * to_end[:, None, :]).float() * kv_scale
    U = torch.matmul((Y * w_end[..., None]).transpose(2, 3), Z)       # [chunks, H, dx, dz]
    seq, off, end = plan["seq"], plan["off"], plan["off"] + plan["length"]
    NC, dx, dz = U.shape[0], U.shape[2], U.shape[3]
    flat = U.permute(1, 0, 2, 3).reshape(H, NC, dx * dz)
    gap = off[:, None] - end[None]
    same = (seq[:, None] == seq[None]) & (gap >= 0)
    D = torch.where(same, torch.exp(gd[:, None, None] * gap.clamp(min=0)), 0.0).float()
    S = torch.matmul(D, flat).reshape(H, NC, dx, dz).transpose(0, 1)
    N = plan["lens"].numel()
    left = plan["lens"][:, None] - end[None]
    mine = seq[None] == torch.arange(N, device=x.device)[:, None]
    E = torch.where(mine, torch.exp(gd[:, None, None] * left.clamp(min=0)), 0.0).float()
    last = torch.matmul(E, flat).reshape(H, N, dx, dz).transpose(0, 1)
    if S_in is not None:
        S = S + torch.exp(off[:, None].double() * gd).float()[..., None, None] * S_in[seq]
        last = last + (torch.exp(plan["lens"][:, None].double() * gd).float()[..., None, None]
                       * S_in)
    first = torch.exp(gd[:, None] * (i[None] + 1 - late)).float()
    out = (out + first[..., None] * torch.matmul(X, S)) * out_scale
    res = torch.zeros(T, H, dz, device=x.device)
    res[idx[valid]] = out.transpose(1, 2)[valid]
    return res, last.contiguous()


def _plain_prefill(s, c):
    o, S = _decayed(s["q"], s["k"], s["v"], s["log_decay"], s["initial_state"], s["plan"], False,
                    c["scale"], 1.0)
    return {"o": o.to(s["q"].dtype), "final_state": S}


def _plain_decode(s, c):
    rows = slice(0, c["B"]) if s["slots"] is None else s["slots"].long()
    S = s["state"][rows] * torch.exp(s["log_decay"])[None, :, None, None]
    S = S + s["k"].float()[..., None] * s["v"].float()[:, :, None, :]
    o = c["scale"] * (S * s["q"].float()[..., None]).sum(dim=2)
    s["state"][rows] = S
    return {"o": o.to(s["q"].dtype), "state": s["state"]}


def _plain_backward(s, c):
    q, k, v, dO, g = s["q"], s["k"], s["v"], s["dO"], s["log_decay"]
    S0, dS = s["initial_state"], s["dS_final"]
    turned = [None if t is None else t.transpose(2, 3) for t in (S0, dS)]
    dq, _ = _decayed(dO, v, k, g, turned[0], s["plan"], False, c["scale"], 1.0)
    dk, _ = _decayed(v, dO, q, g, turned[1], s["plan"], True, 1.0, c["scale"])
    dv, dS0 = _decayed(k, q, dO, g, dS, s["plan"], True, 1.0, c["scale"])
    dt = q.dtype
    return {"dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt), "dS0": dS0}


_EPS = 1e-6


def _gate(t, act):
    return torch.sigmoid(t) if act == "sigmoid" else t * torch.sigmoid(t)


def _plain_norm(s, c):
    T, D = s["y"].shape
    y = s["y"].float().reshape(T, -1, s["w_post"].numel())
    u = y * torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + _EPS) * s["w_post"]
    u = u.reshape(T, D)
    if s["gate"] is not None:
        u = u * _gate(s["gate"].float(), c["gate"])
    if s["res_scale"] is not None:
        u = u * s["res_scale"]
    x = u if s["x"] is None else s["x"].float() + u
    out = {"x_out": x.to(s["y"].dtype)}
    if s["w_pre"] is not None:
        h = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + _EPS) * s["w_pre"]
        out["h"] = h.to(s["y"].dtype)
    return out


def _plain_norm_backward(s, c):
    dt, (T, D) = s["y"].dtype, s["y"].shape
    G = s["w_post"].numel()
    out = {}
    total = s["dx_out"].float()
    if s["w_pre"] is not None:
        x, dh = s["x_out"].float(), s["dh"].float()
        r = torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + _EPS)
        dn = dh * s["w_pre"]
        total = total + r * dn - x * (r ** 3) * (dn * x).mean(dim=-1, keepdim=True)
        out["dw_pre"] = (dh * x * r).sum(dim=0)
    if c["residual"]:
        out["dx"] = total.to(dt)
    y = s["y"].float().reshape(T, -1, G)
    r = torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + _EPS)
    n = (y * r * s["w_post"]).reshape(T, D)
    a = 1.0
    if s["gate"] is not None:
        t = s["gate"].float()
        sig = torch.sigmoid(t)
        a = _gate(t, c["gate"])
        da = sig * (1 - sig) if c["gate"] == "sigmoid" else sig * (1 + t * (1 - sig))
    if s["res_scale"] is not None:
        out["dres_scale"] = (total * n * a).sum(dim=0)
        total = total * s["res_scale"]
    if s["gate"] is not None:
        out["dgate"] = (total * n * da).to(dt)
        total = total * a
    dn = total.reshape(T, -1, G)
    out["dw_post"] = (dn * y * r).sum(dim=(0, 1))
    dn = dn * s["w_post"]
    dy = r * dn - y * (r ** 3) * (dn * y).mean(dim=-1, keepdim=True)
    out["dy"] = dy.reshape(T, D).to(dt)
    return out


_PLAIN = {"lin_prefill": _plain_prefill, "lin_decode": _plain_decode,
          "lin_backward": _plain_backward, "norm": _plain_norm,
          "norm_backward": _plain_norm_backward}


# ------------------------------------------------------- the framework's own
def _own(s, c):
    import kimi_delta_attention_12_gb300 as kda

    op = c["op"]
    if op in ("lin_prefill", "lin_backward"):
        if "workspace" not in s:   # kept by a program between its calls
            size = (kda.lin_prefill_workspace_bytes if op == "lin_prefill"
                    else kda.lin_backward_workspace_bytes)
            s["workspace"] = torch.empty(
                size(len(s["lens"]), s["q"].shape[0], c["H"], c["dk"], c["dv"], s["q"].dtype),
                dtype=torch.uint8, device=s["q"].device)
    if op == "lin_prefill":
        o, S = kda.kda_lin_prefill(s["q"], s["k"], s["v"], s["log_decay"], s["initial_state"],
                                   s["cu"], s["cu_host"], scale=c["scale"],
                                   workspace=s["workspace"])
        return {"o": o, "final_state": S}
    if op == "lin_decode":
        o = kda.kda_lin_decode_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"],
                                    s["slots"], scale=c["scale"])
        return {"o": o, "state": s["state"]}
    if op == "lin_backward":
        return kda.kda_lin_backward(s["q"], s["k"], s["v"], s["log_decay"], s["dO"],
                                    s["initial_state"], s["cu"], s["cu_host"], s["dS_final"],
                                    scale=c["scale"], workspace=s["workspace"])
    if op == "norm":
        x_out, h = kda.kda_block_norm(s["y"], s["w_post"], gate=s["gate"], x=s["x"],
                                      res_scale=s["res_scale"], w_pre=s["w_pre"],
                                      gate_act=c["gate"], eps=_EPS)
        return {"x_out": x_out} if h is None else {"x_out": x_out, "h": h}
    if "workspace" not in s:
        s["workspace"] = torch.empty(
            kda.block_norm_backward_workspace_bytes(*s["y"].shape, s["w_post"].numel()),
            dtype=torch.uint8, device=s["y"].device)
    g = kda.kda_block_norm_backward(s["y"], s["w_post"], s["dx_out"], gate=s["gate"],
                                    x_out=s["x_out"], res_scale=s["res_scale"],
                                    w_pre=s["w_pre"], dh=s["dh"], gate_act=c["gate"], eps=_EPS,
                                    residual=c["residual"], workspace=s["workspace"])
    return {name: t for name, t in g.items() if t is not None}


def run(state):
    c = state["case"]
    return _own(state, c) if own else _PLAIN[c["op"]](state, c)


# ---------------------------------------------------------------------- work
def work(case):
    eb = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("lin_"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        if op == "lin_decode":
            rows = case["B"] * H
            return {"bytes": rows * (2 * dk + 2 * dv) * eb + 2 * rows * dk * dv * 4,
                    "flops": 5 * rows * dk * dv}
        lens = _lens(case)
        pairs, states = sum(lens) * H, len(lens) * H * dk * dv * 4
        if op == "lin_prefill":
            return {"bytes": pairs * (2 * dk + 2 * dv) * eb + states * (2 if case["state"] else 1),
                    "flops": 5 * pairs * dk * dv}
        return {"bytes": pairs * (4 * dk + 3 * dv) * eb + states * (3 if case["state"] else 1),
                "flops": 13 * pairs * dk * dv}
    n, gate = case["rows"] * case["D"], case["gate"] != "none"
    if op == "norm":
        return {"bytes": n * eb * (2 + gate + case["residual"] + case["pre"]), "flops": 12 * n}
    # read y, dx_out, the gate, x_out and dh; write dy, dgate, dx
    return {"bytes": n * eb * (3 + 2 * gate + case["residual"] + 2 * case["pre"]),
            "flops": 30 * n}


# --------------------------------------------------- the definition, 64 bits
def _padded(t, lens):
    """[N, longest, ...] in 64 bits, zeros after each sequence's end."""
    out = torch.zeros(len(lens), max(lens), *t.shape[1:], dtype=torch.float64, device=t.device)
    at = 0
    for n, m in enumerate(lens):
        out[n, :m] = t[at:at + m].double()
        at += m
    return out


def _packed(t, lens):
    return torch.cat([t[n, :m] for n, m in enumerate(lens)])


def _live(lens, t, dev):
    return torch.tensor([float(t < m) for m in lens], dtype=torch.float64,
                        device=dev)[:, None, None, None]


def _exact_forward(q, k, v, a, S, lens, scale):
    """Token by token: S = a S + k v^T, o = scale S^T q; sequences past their end stand still."""
    o = torch.empty(*q.shape[:3], v.shape[-1], dtype=torch.float64, device=q.device)
    ragged = min(lens) < max(lens)
    for t in range(max(lens)):
        new = torch.baddbmm((S * a).flatten(0, 1), k[:, t].flatten(0, 1).unsqueeze(2),
                            v[:, t].flatten(0, 1).unsqueeze(1)).view_as(S)
        S = torch.where(_live(lens, t, q.device) > 0, new, S) if ragged else new
        o[:, t] = scale * torch.matmul(q[:, t].unsqueeze(2), S).squeeze(2)
    return o, S


def exact(case, seed):
    s = _tensors(case, seed)
    op = case["op"]
    if op.startswith("lin_"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        a = torch.exp(s["log_decay"].double())[None, :, None, None]
        if op == "lin_decode":
            rows = torch.arange(case["B"], device=a.device) if s["slots"] is None \
                else s["slots"].long()
            S = s["state"].double()
            S[rows] = S[rows] * a + torch.einsum("bhi,bhj->bhij", s["k"].double(),
                                                 s["v"].double())
            return {"o": case["scale"] * torch.einsum("bhi,bhij->bhj", s["q"].double(), S[rows]),
                    "state": S}
        lens = s["lens"]
        if sum(lens) == 0 or max(lens) * (1 + (op == "lin_backward")) * max(
                1.0, len(lens) * H * dk * dv / 4e6) > 150_000:
            return None
        q, k, v = (_padded(s[n], lens) for n in ("q", "k", "v"))
        zero = torch.zeros(len(lens), H, dk, dv, dtype=torch.float64, device=a.device)
        S0 = zero if s["initial_state"] is None else s["initial_state"].double()
        if op == "lin_prefill":
            o, S = _exact_forward(q, k, v, a, S0, lens, case["scale"])
            return {"o": _packed(o, lens), "final_state": S}
        dO = _padded(s["dO"], lens)
        dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        S = S0
        for t in range(max(lens)):   # dq_t = scale S_t dO_t (what lies past an end is cut off)
            S = S * a + k[:, t, :, :, None] * v[:, t, :, None, :]
            dq[:, t] = case["scale"] * torch.matmul(S, dO[:, t].unsqueeze(3)).squeeze(3)
        G = zero if s["dS_final"] is None else s["dS_final"].double()
        for t in reversed(range(max(lens))):   # G_t = scale q_t dO_t^T + a G_{t+1}
            new = G + case["scale"] * q[:, t, :, :, None] * dO[:, t, :, None, :]
            dk_[:, t] = torch.matmul(new, v[:, t].unsqueeze(3)).squeeze(3)
            dv_[:, t] = torch.matmul(k[:, t].unsqueeze(2), new).squeeze(2)
            G = torch.where(_live(lens, t, q.device) > 0, new * a, G)
        return {"dq": _packed(dq, lens), "dk": _packed(dk_, lens), "dv": _packed(dv_, lens),
                "dS0": G}
    f = {n: t.double().requires_grad_(True) for n, t in s.items()
         if isinstance(t, torch.Tensor) and n not in ("dx_out", "dh")}
    G = s["w_post"].numel()

    def rms(x, w, group):
        blocks = x.unflatten(-1, (-1, group))
        return (blocks / (blocks.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()).flatten(-2) * w

    def branch():
        u = rms(f["y"], f["w_post"].repeat(case["D"] // G), G)
        if "gate" in f:
            u = u * (torch.sigmoid(f["gate"]) if case["gate"] == "sigmoid"
                     else torch.nn.functional.silu(f["gate"]))
        return u * f["res_scale"] if "res_scale" in f else u

    if op == "norm":
        with torch.no_grad():
            x = branch() if "x" not in f else f["x"] + branch()
            out = {"x_out": x}
            if "w_pre" in f:
                out["h"] = rms(x, f["w_pre"], case["D"])
            return out
    # the stream as it was stored stands for x' in the norm before the next block
    total, out = s["dx_out"].double(), {}
    if "w_pre" in f:
        h = rms(f["x_out"], f["w_pre"], case["D"])
        through, out["dw_pre"] = torch.autograd.grad(h, (f["x_out"], f["w_pre"]),
                                                     s["dh"].double())
        total = total + through
    if case["residual"]:
        out["dx"] = total
    names = [n for n in ("y", "w_post", "gate", "res_scale") if n in f]
    grads = torch.autograd.grad(branch(), [f[n] for n in names], total)
    out.update({"d" + n: t for n, t in zip(names, grads)})
    return out
