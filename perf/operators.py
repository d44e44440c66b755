"""Operators of a state-space layer of the serving step, measured case by case.

Four operators, each in a plain torch form and as the library's own call:

* ``scan_decode``: the selective state space step of single tokens (short
  causal convolution, SiLU, gates, state update, readout) over the slot pool;
* ``scan_prefill``: the same recurrence over packed prompts from any start
  position, with block-aligned checkpoints of the state;
* ``add_norm``: the residual addition and RMS norm between the layers, with an
  e4m3 output and its scales for the next projection;
* ``maps``: the packed batch's offsets, block tables, checkpoint table and
  per-token maps, built on the GPU from the requests' lengths.

Formulas (head h of hv reads the q and k of group h // (hv // hk)):
    y = SiLU(conv1d(history, x) + bias);  q, k, v = split(y)
    dt = softplus(a + dt_bias);  S <- exp(-exp(A_log) dt) S + dt v k^T
    o = S q + D v
    h = x + residual;  y = h / sqrt(mean(h^2) + eps) * weight
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"
CHUNK = 64

# layer shapes: (hk, hv, dk, dv, activation type)
SHAPES = {
    "wide": (8, 64, 128, 64, "bf16"),      # 8 groups, 64 heads of 64: a generic state-space layer
    "one": (1, 32, 128, 64, "bf16"),       # a single group read by every head
    "square": (16, 32, 128, 128, "bf16"),  # the heads of the repository's benchmark layer
    "tiny": (2, 4, 16, 16, "f32"),         # the repository's smallest layer, all in fp32
}


def listed():
    return [
        # one user's next token
        dict(name="decode_b1", op="scan_decode", shape="wide", B=1, slots=64, pad=0),
        # an ordinary serving batch with padded rows (a graph captured at a larger batch)
        dict(name="decode_b61_padded", op="scan_decode", shape="wide", B=61, slots=128, pad=5),
        # the largest batch of the benchmark's sweep on the benchmark's heads
        dict(name="decode_b256_square", op="scan_decode", shape="square", B=256, slots=384, pad=0),
        # a short question behind a cached prefix
        dict(name="prefill_1x37", op="scan_prefill", shape="wide", lens="37", starts="320", block=256, slots=8),
        # an agent's turns: odd continuations from unaligned positions, checkpoints every 256 tokens
        dict(name="prefill_ragged", op="scan_prefill", shape="wide", lens="913,1,300,64,2050,129,511",
             starts="0,77,1000,64,0,4095,130", block=256, slots=16),
        # one long document
        dict(name="prefill_1x8192", op="scan_prefill", shape="one", lens="8192", starts="0", block=1024, slots=4),
        # four full prompts, the benchmark's prefill size
        dict(name="prefill_4x8192", op="scan_prefill", shape="wide", lens="8192,8192,8192,8192", starts="0,0,0,0",
             block=1024, slots=8),
        # the smallest layer in fp32
        dict(name="prefill_tiny_f32", op="scan_prefill", shape="tiny", lens="200,33", starts="0,10", block=64, slots=6),
        # the norm before a projection in a decode step, e4m3 with a scale per 128 values
        dict(name="norm_64x4096", op="add_norm", rows=64, d=4096, act="bf16", res="bf16", group=128),
        # the same for a packed prefill, the residual stream kept in fp32, a scale per token
        dict(name="norm_32768x4096_f32res", op="add_norm", rows=32768, d=4096, act="bf16", res="f32", group=0),
        # a decode batch's maps
        dict(name="maps_64", op="maps", n=64, max_len=1, max_start=8192, block=64),
        # many mixed requests
        dict(name="maps_512", op="maps", n=512, max_len=128, max_start=32768, block=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_decode", "scan_prefill", "scan_prefill", "add_norm", "maps"])
    if op == "scan_decode":
        B = _log(rng, 1, 256)
        return dict(op=op, shape=rng.choice(["wide", "one", "square", "tiny"]), B=B, slots=B + rng.randint(1, 64),
                    pad=rng.randint(0, B // 4))
    if op == "scan_prefill":
        shape = rng.choice(["wide", "wide", "one", "square", "tiny"])
        total = _log(rng, 8, 1024 if shape == "tiny" else 8192)
        n = rng.randint(1, min(4 if total > 4096 else 8, total))
        cuts = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        starts = [rng.choice([0, rng.randint(1, 5000)]) for _ in lens]
        return dict(op=op, shape=shape, lens=",".join(map(str, lens)), starts=",".join(map(str, starts)),
                    block=rng.choice([64, 256, 1024]), slots=n + rng.randint(0, 4))
    if op == "add_norm":
        d = 32 * _log(rng, 8, 256)
        return dict(op=op, rows=_log(rng, 1, 16384), d=d, act=rng.choice(["bf16", "bf16", "f32"]),
                    res=rng.choice(["bf16", "f32"]), group=rng.choice([0, 32] + ([128] if d % 128 == 0 else [])))
    return dict(op=op, n=_log(rng, 1, 512), max_len=_log(rng, 1, 128), max_start=_log(rng, 1, 32768),
                block=rng.choice([64, 128, 256]))


# ------------------------------------------------------------------ inputs

def _ints(s):
    return [int(v) for v in s.split(",")]


def _dt(name):
    return BF16 if name == "bf16" else F32


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, shape, std, dtype=F32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _layer(case, g):
    """The layer's weights: step sizes from 1e-3 to 1e-1 before the gate's input, decay rates from 1 to 16."""
    hk, hv, dk, dv, act = SHAPES[case["shape"]]
    C, t = 2 * hk * dk + hv * dv, _dt(act)
    lo, hi = math.log(1e-3), math.log(1e-1)
    dt = torch.exp(torch.rand(hv, generator=g, device=DEV) * (hi - lo) + lo)
    return dict(
        hk=hk, hv=hv, dk=dk, dv=dv, C=C, W=4, act=t,
        conv_w=_normal(g, (C, 4), 0.5), conv_bias=_normal(g, (C,), 0.1),
        A_log=torch.log(1 + 15 * torch.rand(hv, generator=g, device=DEV)),
        dt_bias=dt + torch.log(-torch.expm1(-dt)), D=1 + _normal(g, (hv,), 0.1),
        ssm=_normal(g, (case["slots"], hv, dv, dk), math.sqrt(0.1)),
        conv=_normal(g, (case["slots"], 3, C), math.sqrt(0.1), t))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "scan_decode":
        s = _layer(case, g)
        B = case["B"]
        ids = torch.randperm(case["slots"], generator=g, device=DEV)[:B].to(torch.int32)
        if case["pad"]:
            ids[torch.randperm(B, generator=g, device=DEV)[:case["pad"]]] = -1
        s.update(slot_ids=ids, qkv=_normal(g, (B, s["C"]), 1.0, s["act"]), a=_normal(g, (B, s["hv"]), 1.0, s["act"]),
                 out=torch.zeros((B, s["hv"], s["dv"]), dtype=s["act"], device=DEV))
    elif op == "scan_prefill":
        s = _layer(case, g)
        lens, starts, blk = _ints(case["lens"]), _ints(case["starts"]), case["block"]
        n, total = len(lens), sum(lens)
        cu = [0]
        for v in lens:
            cu.append(cu[-1] + v)
        counts = [(p + v) // blk - p // blk for v, p in zip(lens, starts)]
        mc = max(1, max(counts))
        table = torch.full((n, mc), -1, dtype=torch.int32)
        perm = torch.randperm(sum(counts) + 1, generator=torch.Generator().manual_seed(int(seed))).to(torch.int32)
        at = 0
        for r, c in enumerate(counts):
            table[r, :c] = perm[at:at + c]
            at += c
        s.update(
            total=total, n=n, block=blk, mc=mc,
            # chunks that the longest sequence touches, counted from its first chunk boundary
            nch=max((p % CHUNK + v + CHUNK - 1) // CHUNK for v, p in zip(lens, starts)),
            slot_ids=torch.randperm(case["slots"], generator=g, device=DEV)[:n].to(torch.int32),
            cu=torch.tensor(cu, dtype=torch.int32, device=DEV), start=torch.tensor(starts, dtype=torch.int64, device=DEV),
            ckpt_ids=table.to(DEV), max_len=max(lens),
            ck_ssm=torch.zeros((sum(counts) + 1, s["hv"], s["dv"], s["dk"]), device=DEV),
            ck_conv=torch.zeros((sum(counts) + 1, 3, s["C"]), dtype=s["act"], device=DEV),
            qkv=_normal(g, (total, s["C"]), 1.0, s["act"]), a=_normal(g, (total, s["hv"]), 1.0, s["act"]),
            out=torch.zeros((total, s["hv"], s["dv"]), dtype=s["act"], device=DEV))
    elif op == "add_norm":
        rows, d, group = case["rows"], case["d"], case["group"]
        act, res = _dt(case["act"]), _dt(case["res"])
        s = dict(group=group, eps=1e-6, x=_normal(g, (rows, d), 1.0, act), residual=_normal(g, (rows, d), 2.0, res),
                 weight=1 + _normal(g, (d,), 0.2), y=torch.empty((rows, d), dtype=act, device=DEV),
                 q=torch.empty((rows, d), dtype=torch.float8_e4m3fn, device=DEV),
                 scales=torch.empty((rows, d // (group or d)), device=DEV))
    else:
        n, blk = case["n"], case["block"]
        lens = torch.randint(1, case["max_len"] + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
        start = torch.randint(0, case["max_start"] + 1, (n,), generator=g, device=DEV, dtype=torch.int64)
        mb = (case["max_start"] + case["max_len"]) // blk + 1
        pool = n * (mb + case["max_len"] // blk + 2)
        ids = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
        held = (start + blk - 1) // blk
        col = torch.arange(mb, device=DEV)
        table = torch.where(col < held[:, None], ids[:n * mb].reshape(n, mb), -1).to(torch.int32)
        s = dict(n=n, block=blk, lens=lens, start=start, table=table, max_tokens=n * case["max_len"],
                 free=ids[n * mb:].contiguous(), mc=case["max_len"] // blk + 1)
        s["n_free"] = torch.tensor([s["free"].numel()], dtype=torch.int32, device=DEV)
        s.update(n_free_out=torch.zeros(1, dtype=torch.int32, device=DEV),
                 cu=torch.zeros(n + 1, dtype=torch.int32, device=DEV),
                 ckpt_ids=torch.zeros((n, s["mc"]), dtype=torch.int32, device=DEV),
                 seq_ids=torch.zeros(s["max_tokens"], dtype=torch.int32, device=DEV),
                 positions=torch.zeros(s["max_tokens"], dtype=torch.int64, device=DEV),
                 slot_map=torch.zeros(s["max_tokens"], dtype=torch.int64, device=DEV))
    s["op"] = op
    return s


def _handles(gdn, s):
    """What a program of the library keeps between its calls: the layer's handles and the workspace."""
    if s["op"] in ("scan_decode", "scan_prefill"):
        s["dims"] = gdn.Dims(s["hk"], s["hv"], s["dk"], s["dv"], s["W"], s["act"], s["act"])
        s["pool"] = gdn.StatePool(s["ssm"], s["conv"])
        s["params"] = gdn.SsmParams(s["conv_w"], s["conv_bias"], s["A_log"], s["dt_bias"], s["D"])
    if s["op"] == "scan_prefill":
        s["ckpt"] = gdn.StatePool(s["ck_ssm"], s["ck_conv"])
        size = gdn.ssm_prefill_workspace_size(s["dims"], s["n"], s["total"])
        s["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)
    s["ready"] = True


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    (_own_call if own else {"scan_decode": _plain_decode, "scan_prefill": _plain_prefill, "add_norm": _plain_norm,
                            "maps": _plain_maps}[op])(s)
    if op == "scan_decode":
        return {"out": s["out"], "ssm": s["ssm"], "conv": s["conv"]}
    if op == "scan_prefill":
        return {k: s[k] for k in ("out", "ssm", "conv", "ck_ssm", "ck_conv")}
    if op == "add_norm":
        return {k: s[k] for k in ("residual", "y", "q", "scales")}
    return {k: s[k] for k in ("cu", "table", "ckpt_ids", "seq_ids", "positions", "slot_map", "n_free_out")}


def _own_call(s):
    import hybrid_linear_attention_gdn_gb300 as gdn
    op = s["op"]
    if "ready" not in s:
        _handles(gdn, s)
    if op == "scan_decode":
        gdn.ssm_decode_step(s["dims"], s["pool"], s["params"], s["slot_ids"], s["qkv"], s["a"], s["out"])
    elif op == "scan_prefill":
        gdn.ssm_prefill(s["dims"], s["pool"], s["ckpt"], s["params"], s["slot_ids"], s["cu"], s["start"], s["total"],
                        s["ckpt_ids"], s["block"], s["qkv"], s["a"], s["out"], s["ws"])
    elif op == "add_norm":
        gdn.add_rmsnorm(s["x"], s["residual"], s["weight"], s["eps"], y=s["y"], q8=s["q"], scales=s["scales"],
                        group=s["group"])
    else:
        gdn.batch_maps(s["lens"], s["start"], s["block"], s["table"], s["free"], s["n_free"], s["cu"], s["ckpt_ids"],
                       s["seq_ids"], s["positions"], s["slot_map"], n_free_out=s["n_free_out"])


def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(torch.clamp(x, max=20))))


def _split(s, y):
    """q, k (one row per head) and v of features [..., C]."""
    kd, lead, G = s["hk"] * s["dk"], y.shape[:-1], s["hv"] // s["hk"]
    q = y[..., :kd].reshape(*lead, s["hk"], s["dk"]).repeat_interleave(G, dim=-2)
    k = y[..., kd:2 * kd].reshape(*lead, s["hk"], s["dk"]).repeat_interleave(G, dim=-2)
    return q, k, y[..., 2 * kd:].reshape(*lead, s["hv"], s["dv"])


def _plain_decode(s):
    ids = s["slot_ids"].long()
    live = ids >= 0
    at = ids.clamp(min=0)
    x = torch.cat([s["conv"][at], s["qkv"][:, None]], dim=1)
    y = (x.float() * s["conv_w"].t()).sum(1) + s["conv_bias"]
    q, k, v = _split(s, y / (1 + torch.exp(-y)))
    dt = _softplus(s["a"].float() + s["dt_bias"])
    alpha = torch.exp(-torch.exp(s["A_log"]) * dt)
    S = s["ssm"][at] * alpha[..., None, None] + (dt[..., None] * v)[..., None] * k[..., None, :]
    o = (S * q[..., None, :]).sum(-1) + s["D"][:, None] * v
    s["out"].copy_(torch.where(live[:, None, None], o, torch.zeros_like(o)))
    # padded rows write the slot of the first live row once more, with that row's values
    first = torch.argmax(live.int())
    row = torch.where(live, torch.arange(ids.numel(), device=ids.device), first)
    s["ssm"].index_copy_(0, at[row], S[row])
    s["conv"].index_copy_(0, at[row], x[row, 1:])


def _plain_prefill(s):
    n, T, nch, W = s["n"], CHUNK, s["nch"], s["W"]
    L = nch * T
    ids, cu, p0 = s["slot_ids"].long(), s["cu"].long(), s["start"]
    ln = cu[1:] - cu[:-1]
    # a grid of whole chunks per sequence, aligned to absolute positions
    l = torch.arange(L, device=DEV)[None] - (p0 % T)[:, None]
    inside = (l >= 0) & (l < ln[:, None])
    row = (cu[:-1, None] + l).clamp(0, s["total"] - 1)

    def raw(m):  # the inputs at sequence-relative indices m [n, j]: old history before the first
        x = s["qkv"][(cu[:-1, None] + m).clamp(0, s["total"] - 1)]
        h = s["conv"][ids[:, None], (m + W - 1).clamp(0, W - 2)]
        return torch.where((m >= 0)[..., None], x, h)

    w = s["conv_w"]
    y = s["conv_bias"] + w[:, 3] * raw(l).float() + w[:, 2] * raw(l - 1).float() + w[:, 1] * raw(l - 2).float() \
        + w[:, 0] * raw(l - 3).float()
    y = y / (1 + torch.exp(-y)) * inside[..., None]
    kd, G = s["hk"] * s["dk"], s["hv"] // s["hk"]
    q = y[..., :kd].reshape(n, nch, T, s["hk"], s["dk"])
    k = y[..., kd:2 * kd].reshape(n, nch, T, s["hk"], s["dk"])
    v = y[..., 2 * kd:].reshape(n, nch, T, s["hv"], s["dv"])
    dt = _softplus(s["a"][row].float() + s["dt_bias"]) * inside[..., None]
    g = (-torch.exp(s["A_log"]) * dt).double().reshape(n, nch, T, s["hv"])
    b = g.cumsum(2)                                  # log decay since the chunk's start
    x = dt.reshape(n, nch, T, s["hv"])[..., None] * v
    # each chunk's own state, then all chunks' end states from the earlier chunks' decays
    dS = torch.matmul((x * torch.exp(b[:, :, -1:] - b).float()[..., None]).permute(0, 3, 1, 4, 2),
                      k.permute(0, 3, 1, 2, 4).repeat_interleave(G, dim=1))          # [n, hv, nch, dv, dk]
    e = b[:, :, -1].cumsum(1)                        # [n, nch, hv] log decay since the first chunk's start
    m = (e[:, :, None] - e[:, None]).permute(0, 3, 1, 2)
    tri = torch.ones(nch, nch, dtype=torch.bool, device=DEV).tril()
    m = torch.where(tri, torch.exp(torch.where(tri, m, -torch.inf)), 0).float()      # [n, hv, c, c']
    S0 = s["ssm"][ids]
    end = torch.matmul(m, dS.flatten(3)) + torch.exp(e).float().permute(0, 2, 1)[..., None] * S0.flatten(2)[:, :, None]
    end = end.reshape(n, s["hv"], nch, s["dv"], s["dk"])
    start = torch.cat([S0[:, :, None], end[:, :, :-1]], dim=2)
    # outputs: within the chunk, and from the state that enters it
    low = torch.ones(T, T, dtype=torch.bool, device=DEV).tril()
    bt = b.permute(0, 3, 1, 2)                       # [n, hv, nch, T]
    dec = torch.exp(torch.where(low, bt[..., :, None] - bt[..., None, :], -torch.inf).float())
    qh = q.permute(0, 3, 1, 2, 4)
    qk = torch.matmul(qh, k.permute(0, 3, 1, 4, 2)).repeat_interleave(G, dim=1)
    o = torch.matmul(qk * dec, x.permute(0, 3, 1, 2, 4))
    o = o + torch.exp(bt).float()[..., None] * torch.matmul(qh.repeat_interleave(G, dim=1), start.transpose(-1, -2))
    o = o.permute(0, 2, 3, 1, 4).reshape(n, L, s["hv"], s["dv"]) + (s["D"][:, None] * v).reshape(n, L, s["hv"], s["dv"])
    s["out"][row[inside]] = o[inside].to(s["act"])
    # checkpoints at the block boundaries inside each sequence, then the final state and history
    blk = s["block"]
    P = (p0 // blk * blk)[:, None] + blk * torch.arange(1, s["mc"] + 1, device=DEV)[None]
    has = (P <= (p0 + ln)[:, None]) & (s["ckpt_ids"] >= 0)
    r, c = torch.nonzero(has, as_tuple=True)
    to = s["ckpt_ids"][r, c].long()
    s["ck_ssm"][to] = end[r, :, (P[r, c] // T - p0[r] // T - 1)]
    tail = torch.arange(W - 1, device=DEV) - (W - 1)
    s["ck_conv"][to] = raw(((P - p0[:, None])[:, :, None] + tail).reshape(n, -1)).reshape(n, s["mc"], W - 1, -1)[r, c]
    last = raw(ln[:, None] + tail)
    s["ssm"][ids] = end[:, :, -1]
    s["conv"][ids] = last


def _plain_norm(s):
    h = s["x"].float() + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    rows, d = y.shape
    yg = y.reshape(rows, -1, s["group"] or d)
    top = yg.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / 448, torch.ones_like(top))
    s["residual"].copy_(h)
    s["y"].copy_(y)
    s["q"].copy_((yg / scale).clamp(-448, 448).reshape(rows, d).to(torch.float8_e4m3fn))
    s["scales"].copy_(scale[..., 0])


def _plain_maps(s):
    ln, p0, blk = s["lens"].long(), s["start"], s["block"]
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), ln.cumsum(0)])
    have, need = (p0 + blk - 1) // blk, (p0 + ln + blk - 1) // blk
    base = (need - have).cumsum(0) - (need - have)
    col = torch.arange(s["table"].shape[1], device=DEV)
    fresh = (col >= have[:, None]) & (col < need[:, None])
    k = s["n_free"].long() - 1 - (base[:, None] + col - have[:, None])
    s["table"].copy_(torch.where(fresh, s["free"][k.clamp(0, s["free"].numel() - 1)], s["table"]))
    s["cu"].copy_(cu)
    s["n_free_out"].copy_(s["n_free"] - (need - have).sum())
    c = torch.arange(s["mc"], device=DEV)
    full = (p0 // blk)[:, None] + c
    ok = (full + 1) * blk <= (p0 + ln)[:, None]
    s["ckpt_ids"].copy_(torch.where(ok, s["table"].gather(1, full.clamp(max=s["table"].shape[1] - 1)), -1))
    t = torch.arange(s["max_tokens"], device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    live = seq < s["n"]
    r = seq.clamp(max=s["n"] - 1)
    pos = p0[r] + t - cu[r]
    slot = s["table"][r, (pos // blk).clamp(max=s["table"].shape[1] - 1)].long() * blk + pos % blk
    s["seq_ids"].copy_(torch.where(live, seq, -1))
    s["positions"].copy_(torch.where(live, pos, 0))
    s["slot_map"].copy_(torch.where(live, slot, -1))


# ------------------------------------------------------------------ work and exact values

def work(case):
    op = case["op"]
    if op in ("scan_decode", "scan_prefill"):
        hk, hv, dk, dv, act = SHAPES[case["shape"]]
        e, C, st = (2 if act == "bf16" else 4), 2 * hk * dk + hv * dv, hv * dv * dk
        params = C * 20 + hv * 12
        token = (C + hv + hv * dv) * e
        if op == "scan_decode":
            live = case["B"] - case["pad"]
            return {"bytes": params + live * (8 * st + 6 * C * e + token), "flops": live * (5 * st + 8 * C)}
        lens, starts, blk = _ints(case["lens"]), _ints(case["starts"]), case["block"]
        total = sum(lens)
        ck = sum((p + v) // blk - p // blk for v, p in zip(lens, starts))
        return {"bytes": params + total * token + len(lens) * (8 * st + 6 * C * e) + ck * (4 * st + 3 * C * e),
                "flops": total * (4 * st + 8 * C)}
    if op == "add_norm":
        n = case["rows"] * case["d"]
        a, r = (2 if case["act"] == "bf16" else 4), (2 if case["res"] == "bf16" else 4)
        return {"bytes": n * (a + 2 * r + a + 1) + 4 * case["d"] + 4 * n // (case["group"] or case["d"]),
                "flops": 8 * n}
    n, blk = case["n"], case["block"]
    tokens = n * case["max_len"]
    mc = case["max_len"] // blk + 1
    return {"bytes": n * (12 + 4 + 4 * mc) + 20 * tokens + 8 * (n + tokens // blk), "flops": 4 * tokens}


def exact(case, seed):
    op = case["op"]
    if op == "maps":
        return None
    s = prepare(case, seed)
    if op == "add_norm":
        h = s["x"].double() + s["residual"].double()
        y = s["weight"].double() * h / torch.sqrt(torch.mean(h ** 2, dim=1, keepdim=True) + s["eps"])
        G = s["group"] or y.shape[1]
        peak = y.unflatten(1, (-1, G)).abs().max(dim=2).values
        scale = torch.where(peak == 0, torch.ones_like(peak), peak / 448)
        z = y / scale.repeat_interleave(G, dim=1)
        return {"residual": h, "y": y, "q": _e4m3(z), "scales": scale}
    hk, hv, dk, dv, W = s["hk"], s["hv"], s["dk"], s["dv"], s["W"]
    cw, cb, D = s["conv_w"].double(), s["conv_bias"].double(), s["D"].double()
    rate, bias = torch.exp(s["A_log"].double()), s["dt_bias"].double()
    group = torch.arange(hv, device=DEV) // (hv // hk)

    def step(S, win, a):
        """One token of every row: state S, the window of the last W inputs, the gate's input."""
        y = torch.einsum("nwc,cw->nc", win, cw) + cb
        y = y * torch.sigmoid(y)
        n = y.shape[0]
        q, k, v = y[:, :hk * dk].view(n, hk, dk)[:, group], y[:, hk * dk:2 * hk * dk].view(n, hk, dk)[:, group], \
            y[:, 2 * hk * dk:].view(n, hv, dv)
        dt = torch.nn.functional.softplus(a + bias, threshold=40.0)
        S = torch.exp(-rate * dt)[:, :, None, None] * S + torch.einsum("nhv,nhk->nhvk", dt[:, :, None] * v, k)
        return S, torch.einsum("nhvk,nhk->nhv", S, q) + D[None, :, None] * v

    if op == "scan_decode":
        ssm, conv = s["ssm"].double(), s["conv"].double()
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        live = (s["slot_ids"] >= 0).nonzero()[:, 0]
        ids = s["slot_ids"][live].long()
        win = torch.cat([conv[ids], s["qkv"][live].double()[:, None]], 1)
        ssm[ids], out[live] = step(ssm[ids], win, s["a"][live].double())
        conv[ids] = win[:, 1:]
        return {"out": out, "ssm": ssm, "conv": conv}
    if s["max_len"] > 9000:
        return None
    lens, starts, blk = _ints(case["lens"]), _ints(case["starts"]), case["block"]
    ssm, conv = s["ssm"].double(), s["conv"].double()
    ck_ssm, ck_conv = s["ck_ssm"].double(), s["ck_conv"].double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    order = sorted(range(len(lens)), key=lambda r: -lens[r])  # the rows still running are the first ones
    off = [int(v) for v in s["cu"].tolist()]
    table = s["ckpt_ids"].tolist()
    ids = s["slot_ids"].long()[torch.tensor(order, device=DEV)]
    S, win = ssm[ids], torch.cat([torch.zeros_like(conv[ids][:, :1]), conv[ids]], 1)
    first = torch.tensor([off[r] for r in order], device=DEV)
    for t in range(max(lens)):
        n = sum(lens[r] > t for r in order)
        at = first[:n] + t
        win[:n] = torch.cat([win[:n, 1:], s["qkv"][at].double()[:, None]], 1)
        S[:n], out[at] = step(S[:n], win[:n], s["a"][at].double())
        for j, r in enumerate(order[:n]):
            P = starts[r] + t + 1
            if P % blk == 0:
                c = table[r][P // blk - starts[r] // blk - 1]
                ck_ssm[c], ck_conv[c] = S[j], win[j, 1:]
    ssm[ids], conv[ids] = S, win[:, 1:]
    return {"out": out, "ssm": ssm, "conv": conv, "ck_ssm": ck_ssm, "ck_conv": ck_conv}


def _e4m3(z):
    """Values rounded to the nearest of 4 exponent and 3 mantissa bits (ties to even), at most 448 in magnitude."""
    m = z.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(m.clamp(min=2.0 ** -6)))
    ulp = torch.exp2(e - 3)
    return torch.sign(z) * torch.minimum(torch.round(m / ulp) * ulp, torch.full_like(m, 448.0))
