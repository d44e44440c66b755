"""Operators of a linear-attention layer and of the caches beside it, measured case by case.

Five operators, each in a plain torch form and as the library's own calls:

* ``lin_decode``: linear attention with a fixed decay for each head, one token
  per request, over the slot pool;
* ``lin_prefill``: the same recurrence over packed prompts from any start
  position, with block-aligned checkpoints of the state;
* ``qk_rope``: the norms of queries and keys for each head and the rotation by
  position in one pass, with k and v going to their pages of the cache;
* ``branch``: a request's blocks shared with new branches of it, the partly
  filled last pages copied, the branches given up again;
* ``compact``: the blocks in use moved to the low end of the pool.

Formulas (head h of hv reads the q and k of group h // (hv // hk)):
    S <- exp(log_decay) S + v k^T;  o = scale S q
    y = x / sqrt(mean(x^2) + eps) * weight, then pairs (a, b) -> (a c - b s, b c + a s)
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"
CHUNK = 64

# layer shapes: (hk, hv, dk, dv, activation type)
SHAPES = {
    "heads32": (32, 32, 128, 128, "bf16"),  # a generic layer whose heads all have their own queries and keys
    "grouped": (16, 32, 128, 128, "bf16"),  # the heads of the repository's benchmark layer
    "narrow": (8, 16, 64, 64, "bf16"),      # half the head sizes
    "tiny": (2, 4, 16, 16, "f32"),          # the repository's smallest layer, all in fp32
}


def listed():
    return [
        # one user's next token
        dict(name="lin_decode_b1", op="lin_decode", shape="heads32", B=1, slots=64, pad=0),
        # a large serving batch with padded rows (a graph captured at the benchmark's largest batch)
        dict(name="lin_decode_b256_padded", op="lin_decode", shape="grouped", B=256, slots=300, pad=7),
        # a short question behind a cached prefix
        dict(name="lin_prefill_1x37", op="lin_prefill", shape="grouped", lens="37", starts="320", block=256, slots=8),
        # an agent's turns: odd continuations from unaligned positions, checkpoints every 256 tokens
        dict(name="lin_prefill_ragged", op="lin_prefill", shape="grouped", lens="913,1,300,64,2050,129,511",
             starts="0,77,1000,64,0,4095,130", block=256, slots=16),
        # one long document
        dict(name="lin_prefill_1x8192", op="lin_prefill", shape="heads32", lens="8192", starts="0", block=1024, slots=4),
        # four full prompts, the benchmark's prefill size
        dict(name="lin_prefill_4x8192", op="lin_prefill", shape="heads32", lens="8192,8192,8192,8192",
             starts="0,0,0,0", block=1024, slots=8),
        # a decode batch of an attention layer: 32 query heads over 4 key heads, half of each head rotated
        dict(name="qk_rope_64", op="qk_rope", rows=64, hq=32, hk=4, d=128, rot=64, pairs="halves", act="bf16",
             cache=True, max_pos=32768),
        # a packed prefill of the same layer, all of each head rotated
        dict(name="qk_rope_32768", op="qk_rope", rows=32768, hq=32, hk=4, d=128, rot=128, pairs="halves", act="bf16",
             cache=True, max_pos=32768),
        # four samples of one prompt
        dict(name="branch_1x4", op="branch", parents=1, children=4, max_len=1000, block=64, planes=8, page=16384),
        # four samples each of a batch of long prompts
        dict(name="branch_64x4", op="branch", parents=64, children=4, max_len=8192, block=64, planes=8, page=16384),
        # a small pool with half of its blocks in use
        dict(name="compact_512", op="compact", blocks=512, used=50, rows=32, block=64, planes=8, page=16384),
        # a pool of long use before it is made smaller
        dict(name="compact_8192", op="compact", blocks=8192, used=60, rows=256, block=64, planes=8, page=16384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lin_decode", "lin_prefill", "lin_prefill", "qk_rope", "branch", "compact"])
    if op == "lin_decode":
        B = _log(rng, 1, 256)
        return dict(op=op, shape=rng.choice(list(SHAPES)), B=B, slots=B + rng.randint(1, 64), pad=rng.randint(0, B // 4))
    if op == "lin_prefill":
        shape = rng.choice(["heads32", "grouped", "grouped", "narrow", "tiny"])
        total = _log(rng, 8, 8192 if shape in ("heads32", "grouped") else 2048)
        n = rng.randint(1, min(4 if total > 4096 else 8, total))
        cuts = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        starts = [rng.choice([0, rng.randint(1, 5000)]) for _ in lens]
        return dict(op=op, shape=shape, lens=",".join(map(str, lens)), starts=",".join(map(str, starts)),
                    block=rng.choice([64, 256, 1024]), slots=n + rng.randint(0, 4))
    if op == "qk_rope":
        hk, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        return dict(op=op, rows=_log(rng, 1, 8192), hq=hk * rng.choice([1, 2, 4]), hk=hk, d=d,
                    rot=rng.choice([d, d // 2, d // 4]), pairs=rng.choice(["halves", "halves", "neighbours"]),
                    act=rng.choice(["bf16", "bf16", "f32"]), cache=rng.choice([True, False]),
                    max_pos=_log(rng, 64, 65536))
    if op == "branch":
        return dict(op=op, parents=_log(rng, 1, 48), children=rng.randint(1, 4), max_len=_log(rng, 1, 4096),
                    block=rng.choice([16, 64, 128]), planes=rng.choice([1, 4, 8]), page=256 * _log(rng, 1, 48))
    return dict(op=op, blocks=_log(rng, 16, 4096), used=rng.randint(5, 95), rows=_log(rng, 1, 64), block=64,
                planes=rng.choice([1, 4, 8]), page=256 * _log(rng, 1, 48))


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
    """Decays that forget within 8 tokens in the first head and within 2,000 in the last one."""
    hk, hv, dk, dv, act = SHAPES[case["shape"]]
    C, t = 2 * hk * dk + hv * dv, _dt(act)
    rate = torch.exp(torch.linspace(math.log(1 / 8), math.log(1 / 2000), hv, device=DEV, dtype=torch.float64))
    return dict(hk=hk, hv=hv, dk=dk, dv=dv, C=C, act=t, scale=1 / math.sqrt(dk),
                log_decay=(-rate * torch.exp(0.1 * torch.randn(hv, generator=g, device=DEV))).float(),
                ssm=_normal(g, (case["slots"], hv, dv, dk), 1.0))


def prepare(case, seed):
    g = _gen(seed)
    s = {"lin_decode": _prepare_decode, "lin_prefill": _prepare_prefill, "qk_rope": _prepare_rope,
         "branch": _prepare_branch, "compact": _prepare_compact}[case["op"]](case, g)
    s["op"] = case["op"]
    return s


def _prepare_decode(case, g):
    s = _layer(case, g)
    B = case["B"]
    ids = torch.randperm(case["slots"], generator=g, device=DEV)[:B].to(torch.int32)
    if case["pad"]:
        ids[torch.randperm(B, generator=g, device=DEV)[:case["pad"]]] = -1
    s.update(slot_ids=ids, qkv=_normal(g, (B, s["C"]), 1.0, s["act"]),
             out=torch.zeros((B, s["hv"], s["dv"]), dtype=s["act"], device=DEV))
    return s


def _prepare_prefill(case, g):
    s = _layer(case, g)
    lens, starts, blk = _ints(case["lens"]), _ints(case["starts"]), case["block"]
    n, total = len(lens), sum(lens)
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    counts = [(p + v) // blk - p // blk for v, p in zip(lens, starts)]
    mc = max(1, max(counts))
    table = torch.full((n, mc), -1, dtype=torch.int32, device=DEV)
    perm = torch.randperm(sum(counts) + 1, generator=g, device=DEV).to(torch.int32)
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
        ckpt_ids=table, ck_ssm=torch.zeros((sum(counts) + 1, s["hv"], s["dv"], s["dk"]), device=DEV),
        qkv=_normal(g, (total, s["C"]), 1.0, s["act"]),
        out=torch.zeros((total, s["hv"], s["dv"]), dtype=s["act"], device=DEV))
    return s


def _prepare_rope(case, g):
    rows, hq, hk, d, rot, t = case["rows"], case["hq"], case["hk"], case["d"], case["rot"], _dt(case["act"])
    # the projection's rows: q | k | v
    x = _normal(g, (rows, (hq + 2 * hk) * d), 1.0, t)
    # the angles of every position, cosines then sines
    f = 1e6 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2 / rot)
    ang = torch.arange(case["max_pos"], device=DEV, dtype=torch.float64)[:, None] * f
    s = dict(q=x[:, :hq * d].view(rows, hq, d), k=x[:, hq * d:(hq + hk) * d].view(rows, hk, d),
             v=x[:, (hq + hk) * d:].view(rows, hk, d), eps=1e-6, pairs=case["pairs"], rot=rot, cache=case["cache"],
             q_weight=1 + _normal(g, (d,), 0.2), k_weight=1 + _normal(g, (d,), 0.2),
             cos_sin=torch.cat([torch.cos(ang), torch.sin(ang)], 1).float(),
             positions=torch.randint(0, case["max_pos"], (rows,), generator=g, device=DEV),
             q_out=torch.zeros((rows, hq, d), dtype=t, device=DEV))
    if case["cache"]:
        # pages of 64 rows; some rows of the batch are padding
        pages = (rows + 63) // 64 + 4
        slot = torch.randperm(pages * 64, generator=g, device=DEV)[:rows]
        s["slot_map"] = torch.where(torch.rand(rows, generator=g, device=DEV) < 0.03, -1, slot)
        s["k_cache"] = torch.zeros((pages, 64, hk, d), dtype=t, device=DEV)
        s["v_cache"] = torch.zeros((pages, 64, hk, d), dtype=t, device=DEV)
    else:
        s["k_out"] = torch.zeros((rows, hk, d), dtype=t, device=DEV)
    return s


def _planes(case, blocks, g):
    return [torch.randn((blocks, case["page"] // 2), generator=g, device=DEV, dtype=BF16) for _ in range(case["planes"])]


def _prepare_branch(case, g):
    P, c, blk = case["parents"], case["children"], case["block"]
    lens = torch.randint((case["max_len"] + 1) // 2, case["max_len"] + 1, (P,), generator=g, device=DEV)
    mb = (case["max_len"] + blk - 1) // blk
    n = P * c
    blocks = P * mb + n
    ids = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    table = torch.full((P + n, mb), -1, dtype=torch.int32, device=DEV)
    held = ((lens + blk - 1) // blk)[:, None] > torch.arange(mb, device=DEV)
    table[:P] = torch.where(held, ids[:P * mb].view(P, mb), -1)
    src = torch.arange(P, device=DEV, dtype=torch.int32).repeat_interleave(c)
    i32 = dict(dtype=torch.int32, device=DEV)
    s = dict(n=n, block=blk, blocks=blocks, table=table, src_rows=src, dst_rows=torch.arange(P, P + n, **i32),
             lens=lens[src.long()].contiguous(), none=torch.zeros(n, dtype=torch.int64, device=DEV),
             refs=torch.zeros(blocks, **i32), free=torch.cat([ids[P * mb:], torch.full((P * mb,), -1, **i32)]),
             n_free=torch.full((1,), n, **i32), copy_src=torch.zeros(n, **i32), copy_dst=torch.zeros(n, **i32),
             child_table=torch.zeros((n, mb), **i32), planes=_planes(case, blocks, g))
    return s


def _prepare_compact(case, g):
    N, R = case["blocks"], case["rows"]
    live = max(1, N * case["used"] // 100)
    ids = torch.randperm(N, generator=g, device=DEV).to(torch.int32)
    # the blocks in use, a few of them held by two requests
    mb = (live + R - 1) // R + 2
    table = torch.full((R, mb), -1, dtype=torch.int32, device=DEV)
    at = torch.arange(live, device=DEV)
    table[at % R, at // R] = ids[:live]
    share = torch.rand(R, generator=g, device=DEV) < 0.5
    table[:, mb - 1] = torch.where(share, table[:, 0].roll(1), -1)
    held = torch.zeros(N + 1, dtype=torch.int32, device=DEV)
    held.index_add_(0, torch.where(table < 0, N, table).long().flatten(), torch.ones(R * mb, dtype=torch.int32, device=DEV))
    i32 = dict(dtype=torch.int32, device=DEV)
    s = dict(table=table, refs=(held[:N] - 1).clamp(min=0), blocks=N,
             free=torch.cat([ids[live:], torch.full((live,), -1, **i32)]), n_free=torch.full((1,), N - live, **i32),
             table_out=torch.zeros((R, mb), **i32), refs_out=torch.zeros(N, **i32), free_out=torch.zeros(N, **i32),
             move_src=torch.zeros(N // 2 + 1, **i32), move_dst=torch.zeros(N // 2 + 1, **i32),
             n_moves=torch.zeros(1, **i32), planes=_planes(case, N, g))
    return s


def _handles(gdn, s):
    """What a program of the library keeps between its calls: the layer's handles, the workspaces, the planes."""
    if s["op"] in ("lin_decode", "lin_prefill"):
        s["dims"] = gdn.Dims(s["hk"], s["hv"], s["dk"], s["dv"], 1, s["act"], s["act"])
        s["pool"] = gdn.StatePool(s["ssm"])
    if s["op"] == "lin_prefill":
        s["ckpt"] = gdn.StatePool(s["ck_ssm"])
        size = gdn.lin_prefill_workspace_size(s["dims"], s["n"], s["total"])
        s["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)
    if s["op"] in ("branch", "compact"):
        s["cache"] = gdn.PagePlanes(s["planes"])
    if s["op"] == "compact":
        s["ws"] = torch.empty(gdn.block_compact_workspace_size(s["blocks"]), dtype=torch.uint8, device=DEV)
    s["ready"] = True


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    (_own_call if own else {"lin_decode": _plain_decode, "lin_prefill": _plain_prefill, "qk_rope": _plain_rope,
                            "branch": _plain_branch, "compact": _plain_compact}[op])(s)
    if op == "lin_decode":
        return {"out": s["out"], "ssm": s["ssm"]}
    if op == "lin_prefill":
        return {k: s[k] for k in ("out", "ssm", "ck_ssm")}
    if op == "qk_rope":
        return {k: s[k] for k in ("q_out",) + (("k_cache", "v_cache") if s["cache"] else ("k_out",))}
    if op == "branch":
        return {k: s[k] for k in ("child_table", "table", "copy_src", "copy_dst", "refs", "free", "n_free", "planes")}
    return {k: s[k] for k in ("table_out", "refs_out", "free_out", "move_src", "move_dst", "n_moves", "planes")}


def _own_call(s):
    import hybrid_linear_attention_gdn_gb300 as gdn
    op = s["op"]
    if "ready" not in s:
        _handles(gdn, s)
    if op == "lin_decode":
        gdn.lin_decode_step(s["dims"], s["pool"], s["log_decay"], s["slot_ids"], s["qkv"], s["out"], scale=s["scale"])
    elif op == "lin_prefill":
        gdn.lin_prefill(s["dims"], s["pool"], s["ckpt"], s["log_decay"], s["slot_ids"], s["cu"], s["start"], s["total"],
                        s["ckpt_ids"], s["block"], s["qkv"], s["out"], s["ws"], scale=s["scale"])
    elif op == "qk_rope":
        gdn.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["cos_sin"], s["positions"], eps=s["eps"],
                         interleaved=s["pairs"] == "neighbours", q_out=s["q_out"], k_out=s.get("k_out"),
                         v=s["v"] if s["cache"] else None, k_cache=s.get("k_cache"), v_cache=s.get("v_cache"),
                         slot_map=s.get("slot_map"))
    elif op == "branch":
        gdn.block_fork(s["src_rows"], s["dst_rows"], s["lens"], s["block"], s["table"], s["refs"], s["free"],
                       s["n_free"], s["copy_src"], s["copy_dst"])
        gdn.page_copy(s["cache"], s["copy_src"], s["copy_dst"])
        s["child_table"].copy_(s["table"][-s["n"]:])
        gdn.block_release(s["dst_rows"], s["lens"], s["none"], s["block"], s["table"], s["refs"], s["free"],
                          s["n_free"])
    else:
        gdn.block_compact(s["table"], s["refs"], s["free"], s["n_free"], s["move_src"], s["move_dst"], s["n_moves"],
                          s["ws"], table_out=s["table_out"], refs_out=s["refs_out"], free_out=s["free_out"])
        gdn.page_copy(s["cache"], s["move_src"], s["move_dst"])


def _split(s, x):
    """q, k (one row per head) and v of rows [..., C], in fp32."""
    kd, lead, G = s["hk"] * s["dk"], x.shape[:-1], s["hv"] // s["hk"]
    x = x.float()
    q = x[..., :kd].reshape(*lead, s["hk"], s["dk"]).repeat_interleave(G, dim=-2)
    k = x[..., kd:2 * kd].reshape(*lead, s["hk"], s["dk"]).repeat_interleave(G, dim=-2)
    return q, k, x[..., 2 * kd:].reshape(*lead, s["hv"], s["dv"])


def _plain_decode(s):
    ids = s["slot_ids"].long()
    live = ids >= 0
    at = ids.clamp(min=0)
    q, k, v = _split(s, s["qkv"])
    S = s["ssm"][at] * torch.exp(s["log_decay"])[:, None, None] + v[..., None] * k[..., None, :]
    o = (S * q[..., None, :]).sum(-1) * s["scale"]
    s["out"].copy_(torch.where(live[:, None, None], o, torch.zeros_like(o)))
    # padded rows write the slot of the first live row once more, with that row's values
    first = torch.argmax(live.int())
    row = torch.where(live, torch.arange(ids.numel(), device=ids.device), first)
    s["ssm"].index_copy_(0, at[row], S[row])


def _plain_prefill(s):
    n, T, nch = s["n"], CHUNK, s["nch"]
    L = nch * T
    ids, cu, p0 = s["slot_ids"].long(), s["cu"].long(), s["start"]
    ln = cu[1:] - cu[:-1]
    # a grid of whole chunks per sequence, aligned to absolute positions; rows outside have k = 0 and no decay
    l = torch.arange(L, device=DEV)[None] - (p0 % T)[:, None]
    inside = (l >= 0) & (l < ln[:, None])
    row = (cu[:-1, None] + l).clamp(0, s["total"] - 1)
    hv, hk, G = s["hv"], s["hk"], s["hv"] // s["hk"]
    kd = hk * s["dk"]
    x = s["qkv"][row].float() * inside[..., None]
    q = x[..., :kd].reshape(n, nch, T, hk, s["dk"]).permute(0, 3, 1, 2, 4)           # [n, hk, nch, T, dk]
    k = x[..., kd:2 * kd].reshape(n, nch, T, hk, s["dk"]).permute(0, 3, 1, 2, 4)
    v = x[..., 2 * kd:].reshape(n, nch, T, hv, s["dv"]).permute(0, 3, 1, 2, 4)        # [n, hv, nch, T, dv]
    g = s["log_decay"].double()[None, :, None, None] * inside.reshape(n, 1, nch, T)
    b = g.cumsum(3)                                                                   # log decay since the chunk's start
    kh, qh = k.repeat_interleave(G, dim=1), q.repeat_interleave(G, dim=1)
    # each chunk's own state, then all chunks' end states from the earlier chunks' decays
    dS = torch.matmul((v * torch.exp(b[..., -1:] - b).float()[..., None]).transpose(-1, -2), kh)
    e = b[..., -1].cumsum(2)                                                          # [n, hv, nch]
    tri = torch.ones(nch, nch, dtype=torch.bool, device=DEV).tril()
    m = torch.exp(torch.where(tri, e[..., :, None] - e[..., None, :], -torch.inf)).float()
    S0 = s["ssm"][ids]
    end = torch.matmul(m, dS.flatten(3)) + torch.exp(e).float()[..., None] * S0.flatten(2)[:, :, None]
    end = end.reshape(n, hv, nch, s["dv"], s["dk"])
    start = torch.cat([S0[:, :, None], end[:, :, :-1]], dim=2)
    # outputs: within the chunk, and from the state that enters it
    low = torch.ones(T, T, dtype=torch.bool, device=DEV).tril()
    dec = torch.exp(torch.where(low, b[..., :, None] - b[..., None, :], -torch.inf).float())
    qk = torch.matmul(q, k.transpose(-1, -2)).repeat_interleave(G, dim=1)
    o = torch.matmul(qk * dec, v) + torch.exp(b).float()[..., None] * torch.matmul(qh, start.transpose(-1, -2))
    o = (o * s["scale"]).permute(0, 2, 3, 1, 4).reshape(n, L, hv, s["dv"])
    s["out"][row[inside]] = o[inside].to(s["act"])
    # checkpoints at the block boundaries inside each sequence, then the final state
    blk = s["block"]
    P = (p0 // blk * blk)[:, None] + blk * torch.arange(1, s["mc"] + 1, device=DEV)[None]
    r, c = torch.nonzero((P <= (p0 + ln)[:, None]) & (s["ckpt_ids"] >= 0), as_tuple=True)
    s["ck_ssm"][s["ckpt_ids"][r, c].long()] = end[r, :, P[r, c] // T - p0[r] // T - 1]
    s["ssm"][ids] = end[:, :, -1]


def _plain_rope(s):
    cs = s["cos_sin"][s["positions"]]
    half = s["rot"] // 2
    c, n = cs[:, None, :half], cs[:, None, half:]

    def turn(x, w):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w
        head, rest = y[..., :s["rot"]], y[..., s["rot"]:]
        if s["pairs"] == "halves":
            a, b = head[..., :half], head[..., half:]
            return torch.cat([a * c - b * n, b * c + a * n, rest], -1)
        a, b = head[..., 0::2], head[..., 1::2]
        return torch.cat([torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2), rest], -1)

    s["q_out"].copy_(turn(s["q"], s["q_weight"]))
    k = turn(s["k"], s["k_weight"])
    if not s["cache"]:
        s["k_out"].copy_(k)
        return
    # padded rows write the slot of the first live row once more, with that row's values
    live = s["slot_map"] >= 0
    row = torch.where(live, torch.arange(live.numel(), device=DEV), torch.argmax(live.int()))
    at = torch.where(live.any(), s["slot_map"][row], 0)
    for cache, x in ((s["k_cache"].flatten(0, 1), k.to(s["k_cache"].dtype)), (s["v_cache"].flatten(0, 1), s["v"])):
        cache.index_copy_(0, at, torch.where(live.any(), x[row], cache[at]))


def _plain_copy(planes, src, dst):
    # pairs of -1 copy the page of the first pair once more
    live = src >= 0
    pair = torch.where(live, torch.arange(live.numel(), device=DEV), torch.argmax(live.int()))
    a, b = src[pair].long().clamp(min=0), dst[pair].long().clamp(min=0)
    b = torch.where(live.any(), b, a)
    for p in planes:
        p.index_copy_(0, b, p[a])


def _plain_branch(s):
    blk, t = s["block"], s["table"]
    src, dst = s["src_rows"].long(), s["dst_rows"].long()
    col = torch.arange(t.shape[1], device=DEV)
    full, part = s["lens"] // blk, s["lens"] % blk > 0
    rank = part.cumsum(0) - 1
    new = s["free"][torch.where(part, s["n_free"].long() - 1 - rank, 0)]
    shared = col < full[:, None]
    rows = t[src]
    last = part[:, None] & (col == full[:, None])
    t[dst] = torch.where(shared, rows, torch.where(last, new[:, None], t[dst]))
    s["refs"].index_add_(0, torch.where(shared, rows, 0).long().flatten(), shared.int().flatten())
    s["copy_src"].copy_(torch.where(part, rows.gather(1, full.clamp(max=t.shape[1] - 1)[:, None])[:, 0], -1))
    s["copy_dst"].copy_(torch.where(part, new, -1))
    s["n_free"].sub_(part.sum())
    _plain_copy(s["planes"], s["copy_src"], s["copy_dst"])
    s["child_table"].copy_(t[-s["n"]:])
    # the branches are given up: blocks that nobody else holds go onto the stack, by id
    first, held = (s["none"] + blk - 1) // blk, (s["lens"] + blk - 1) // blk
    gone = (col >= first[:, None]) & (col < held[:, None])
    rows = t[dst]
    s["refs"].index_add_(0, torch.where(gone, rows, 0).long().flatten(), -gone.int().flatten())
    t[dst] = torch.where(gone, -1, rows)
    free = s["refs"] < 0
    s["refs"].clamp_(min=0)
    at = torch.where(free, s["n_free"].long() + free.cumsum(0) - 1, s["blocks"])
    s["free"].copy_(torch.cat([s["free"], s["free"][:1]]).scatter_(
        0, at, torch.arange(s["blocks"], device=DEV, dtype=torch.int32))[:-1])
    s["n_free"].add_(free.sum())


def _plain_compact(s):
    N, dev = s["blocks"], dict(device=DEV)
    nf = s["n_free"].long()
    ids = torch.arange(N, **dev)
    slot = torch.where(ids < nf, s["free"].long(), N)
    free = torch.zeros(N + 1, dtype=torch.bool, **dev).scatter_(0, slot, True)[:N]
    live = N - nf
    # the k-th highest block in use above the border goes to the k-th lowest free one below it
    mover, hole = ~free & (ids >= live), free & (ids < live)
    M = s["move_src"].numel()
    up = mover.flip(0).cumsum(0).flip(0) - 1
    down = hole.cumsum(0) - 1
    src = torch.full((M + 1,), -1, dtype=torch.int32, **dev)
    src.scatter_(0, torch.where(mover, up, M), torch.where(mover, ids, -1).int())
    dst = torch.full((M + 1,), -1, dtype=torch.int32, **dev)
    dst.scatter_(0, torch.where(hole, down, M), torch.where(hole, ids, -1).int())
    s["move_src"].copy_(src[:M])
    s["move_dst"].copy_(dst[:M])
    s["n_moves"].copy_(mover.sum())
    to = torch.where(mover, dst[torch.where(mover, up, M)].long(), ids)
    t = s["table"].long()
    s["table_out"].copy_(torch.where(t >= 0, to[t.clamp(min=0)], t))
    refs = torch.where(ids < live, s["refs"], 0)
    s["refs_out"].copy_(torch.cat([refs, refs[:1]]).scatter_(0, torch.where(mover, to, N), s["refs"])[:N])
    # the free ids are the high ones, the lowest of them on top; what lies above the stack's top stays
    s["free_out"].copy_(torch.where(ids < nf, N - 1 - ids, s["free"]))
    _plain_copy(s["planes"], s["move_src"], s["move_dst"])


# ------------------------------------------------------------------ work and exact values

def work(case):
    op = case["op"]
    if op in ("lin_decode", "lin_prefill"):
        hk, hv, dk, dv, act = SHAPES[case["shape"]]
        e, C, st = (2 if act == "bf16" else 4), 2 * hk * dk + hv * dv, hv * dv * dk
        token = (C + hv * dv) * e
        if op == "lin_decode":
            live = case["B"] - case["pad"]
            return {"bytes": hv * 4 + live * (8 * st + token), "flops": live * 5 * st}
        lens, starts, blk = _ints(case["lens"]), _ints(case["starts"]), case["block"]
        ck = sum((p + v) // blk - p // blk for v, p in zip(lens, starts))
        return {"bytes": hv * 4 + sum(lens) * token + len(lens) * 8 * st + ck * 4 * st, "flops": sum(lens) * 4 * st}
    if op == "qk_rope":
        e, rows = (2 if case["act"] == "bf16" else 4), case["rows"]
        heads = case["hq"] + case["hk"] * (2 if case["cache"] else 1)
        return {"bytes": rows * (2 * heads * case["d"] * e + case["rot"] * 4 + 8 + (8 if case["cache"] else 0)),
                "flops": rows * (case["hq"] + case["hk"]) * case["d"] * 8}
    if op == "branch":
        n = case["parents"] * case["children"]
        held = (case["max_len"] * 3 // 4 + case["block"] - 1) // case["block"]
        return {"bytes": n * (2 * case["planes"] * case["page"] + held * 24 + 40), "flops": n * held}
    N, live = case["blocks"], max(1, case["blocks"] * case["used"] // 100)
    moves = live * (N - live) // N
    return {"bytes": moves * (2 * case["planes"] * case["page"] + 8) + N * 16 + live * 8, "flops": N}


def exact(case, seed):
    op = case["op"]
    if op in ("branch", "compact"):
        return None
    s = prepare(case, seed)
    if op == "qk_rope":
        return _exact_rope(s)
    hk, hv, dk, dv = s["hk"], s["hv"], s["dk"], s["dv"]
    group = torch.arange(hv, device=DEV) // (hv // hk)
    keep = torch.exp(s["log_decay"].double())[:, None, None]
    x = s["qkv"]
    q, k, v = x[:, :hk * dk], x[:, hk * dk:2 * hk * dk], x[:, 2 * hk * dk:]

    def step(S, at):
        """One token of every row: state S and the token's row in the batch."""
        qt, kt = q[at].double().view(-1, hk, dk)[:, group], k[at].double().view(-1, hk, dk)[:, group]
        S = torch.einsum("nhv,nhk->nhvk", v[at].double().view(-1, hv, dv), kt) + keep * S
        return S, s["scale"] * torch.einsum("nhvk,nhk->nhv", S, qt)

    ssm, out = s["ssm"].double(), torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    if op == "lin_decode":
        live = (s["slot_ids"] >= 0).nonzero()[:, 0]
        ids = s["slot_ids"][live].long()
        ssm[ids], out[live] = step(ssm[ids], live)
        return {"out": out, "ssm": ssm}
    lens, starts, blk = _ints(case["lens"]), _ints(case["starts"]), case["block"]
    if max(lens) > 9000:
        return None
    ck = s["ck_ssm"].double()
    order = sorted(range(len(lens)), key=lambda r: -lens[r])  # the rows still running are the first ones
    off, table = s["cu"].tolist(), s["ckpt_ids"].tolist()
    ids = s["slot_ids"].long()[torch.tensor(order, device=DEV)]
    S = ssm[ids]
    first = torch.tensor([off[r] for r in order], device=DEV)
    for t in range(max(lens)):
        n = sum(lens[r] > t for r in order)
        at = first[:n] + t
        S[:n], out[at] = step(S[:n], at)
        for j, r in enumerate(order[:n]):
            P = starts[r] + t + 1
            if P % blk == 0:
                ck[table[r][P // blk - starts[r] // blk - 1]] = S[j]
    ssm[ids] = S
    return {"out": out, "ssm": ssm, "ck_ssm": ck}


def _exact_rope(s):
    half, tab = s["rot"] // 2, s["cos_sin"].double()[s["positions"]]
    # each pair as a complex number, turned by multiplication
    turn = torch.complex(tab[:, :half], tab[:, half:])[:, None]

    def head(x, w):
        x = x.double()
        y = x / torch.sqrt(torch.mean(x ** 2, dim=2, keepdim=True) + s["eps"]) * w.double()
        z = y.clone()
        lo, hi = (slice(0, half), slice(half, 2 * half)) if s["pairs"] == "halves" \
            else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
        p = torch.complex(y[..., lo], y[..., hi]) * turn
        z[..., lo], z[..., hi] = p.real, p.imag
        return z

    q, k = head(s["q"], s["q_weight"]), head(s["k"], s["k_weight"])
    if not s["cache"]:
        return {"q_out": q, "k_out": k}
    live = (s["slot_map"] >= 0).nonzero()[:, 0]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    at = s["slot_map"][live]
    kc.view(-1, *k.shape[1:])[at], vc.view(-1, *k.shape[1:])[at] = k[live], s["v"][live].double()
    return {"q_out": q, "k_cache": kc, "v_cache": vc}
