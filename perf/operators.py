"""Cases of the attention operators over parts of the sequence: block selection, attention over the selected
blocks, appending keys and values to a paged cache, and attention of new tokens over that cache.

``run`` computes them in plain torch operations, or (``own``) through the package's binding.
"""
import math

import torch

own = False

HD = 128  # head width of every Wan model
EPS = 1e-6
THETA = 10000.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one block of the CPU-sized model: 3x8x8 tokens, the cheapest selection
        _select("select 192 tokens", 1, 12, (3, 8, 8), (3, 8, 8), (1, 8, 8), (1, 4, 4), 6, False),
        # the 480p 81-frame step with guidance (two samples), an eighth of the key blocks kept
        _select("select 480p pair", 2, 12, (21, 30, 52), (21, 30, 52), (4, 4, 8), (4, 4, 4), 78, False),
        # a 720p 81-frame step of the 14B model, the first blocks always kept and far frames never
        _select("select 720p 14B masked", 1, 40, (21, 45, 80), (21, 45, 80), (4, 4, 8), (4, 4, 8), 96, True),
        # the small model again, uneven lists and rows without any block
        _blocks("blocks 192 tokens", 2, 12, (3, 8, 8), (3, 8, 8), (1, 8, 8), (1, 4, 4), 6, True),
        # one latent frame of queries against 21 frames of keys (chunked generation): few query blocks
        _blocks("blocks frame on window", 1, 12, (1, 30, 52), (21, 30, 52), (1, 8, 16), (1, 8, 8), 147, False),
        # the 480p 81-frame self-attention, an eighth of the key blocks
        _blocks("blocks 480p", 1, 12, (21, 30, 52), (21, 30, 52), (4, 4, 8), (4, 4, 4), 78, False),
        # one new token (an action or state token) for each of 16 streams
        _append("append one token", 16, 1, 12, (30, 52), 64, 21, False, False),
        # three latent frames of a 480p stream: the packed q, k, v rows of one chunk
        _append("append chunk 480p", 1, 4680, 12, (30, 52), 64, 24, True, False),
        # ragged chunks of four 14B streams, 128-token pages
        _append("append ragged 14B", 4, 1560, 40, (30, 52), 128, 6, True, True),
        # one new token on a cache of 84 latent frames
        _paged("paged one token", 1, 1, 12, 131040, 64, False),
        # one new token for each of 16 streams of different lengths, small pages
        _paged("paged ragged tokens", 16, 1, 12, 16380, 16, True),
        # one latent frame of queries over 21 cached frames
        _paged("paged frame", 1, 1560, 12, 32760, 64, False),
    ]


def _select(name, B, heads, qg, kg, qb, kb, topk, masked):
    return _geometry({"name": name, "op": "select", "B": B, "heads": heads, "topk": topk, "masked": masked}, qg, kg, qb, kb)


def _blocks(name, B, heads, qg, kg, qb, kb, topk, ragged):
    return _geometry({"name": name, "op": "blocks", "B": B, "heads": heads, "topk": topk, "ragged": ragged}, qg, kg, qb, kb)


def _append(name, B, T, heads, hw, page, frames, norm, ragged):
    return {"name": name, "op": "append", "B": B, "T": T, "heads": heads, "H": hw[0], "W": hw[1], "page": page,
            "frames": frames, "norm": norm, "ragged": ragged}


def _paged(name, B, T, heads, length, page, ragged):
    return {"name": name, "op": "paged", "B": B, "T": T, "heads": heads, "length": length, "page": page, "ragged": ragged}


def _geometry(case, qg, kg, qb, kb):
    for key, dims in (("qg", qg), ("kg", kg), ("qb", qb), ("kb", kb)):
        for axis, n in zip("FHW", dims):
            case[key + axis] = n
    return case


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["select", "blocks", "append", "paged"])
    heads = rng.choice([1, 3, 5, 8, 12, 12, 16, 20])
    if op in ("select", "blocks"):
        heads = min(heads, 12)
        kg = (log(1, 21), log(2, 32), log(2, 54))
        if op == "select":  # something to choose from
            heads, kg = max(heads, 3), (log(4, 21), log(8, 32), log(24, 54))
        qg = kg if rng.random() < 0.7 else (log(1, kg[0]), kg[1], kg[2])
        qb = rng.choice([(4, 4, 8), (1, 8, 16), (2, 8, 8), (1, 8, 8), (4, 4, 4), (3, 5, 7)])
        kb = rng.choice([(4, 4, 4), (1, 8, 8), (4, 4, 8), (2, 8, 8), (2, 4, 4), (1, 4, 4)])
        if rng.random() < 0.15:  # one token axis, as text is
            kg = qg = (1, 1, log(1024 if op == "select" else 1, 16384))
            qb, kb = (1, 1, 128), (1, 1, rng.choice([64, 128]))
        nk = _count(kg, kb)
        topk = min(nk, log(1, max(1, nk // 6 + 1)), 9984 // (kb[0] * kb[1] * kb[2]))
        make = _select if op == "select" else _blocks
        B = rng.choice([1, 1, 2]) if op == "select" else 1
        case = make("", B, heads, qg, kg, qb, kb, max(1, topk), rng.random() < 0.4)
    elif op == "append":
        hw = (log(1, 45), log(1, 80))
        frames = log(1, 24)
        most = max(1, min(frames * hw[0] * hw[1], 6000))
        B = log(1, 16)
        T = log(1, max(1, most // B))
        case = _append("", B, T, heads, hw, rng.choice([16, 32, 64, 128]), frames, rng.random() < 0.6, rng.random() < 0.5)
    else:
        B = log(1, 16)
        T = log(1, 1600 // B) if rng.random() < 0.6 else 1
        length = log(max(1, T), max(T + 1, 131040 // B if T == 1 else 32760 // B))
        case = _paged("", B, T, heads, length, rng.choice([16, 32, 64, 128]), rng.random() < 0.5)
    del case["name"]
    return case


# ---------------------------------------------------------------- geometry
def _grid(case, key):
    return tuple(case[key + a] for a in "FHW")


def _volume(b):
    return b[0] * b[1] * b[2]


def _numbers(grid, block):
    return tuple(-(-g // b) for g, b in zip(grid, block))


def _count(grid, block):
    return _volume(_numbers(grid, block))


def _tokens(grid, block, device):
    """Token number of each place of each block [blocks, volume], and whether the place is inside the grid."""
    n = _numbers(grid, block)
    axes = [torch.arange(n[a], device=device)[:, None] * block[a] + torch.arange(block[a], device=device) for a in range(3)]
    f = axes[0].view(n[0], 1, 1, block[0], 1, 1)
    i = axes[1].view(1, n[1], 1, 1, block[1], 1)
    j = axes[2].view(1, 1, n[2], 1, 1, block[2])
    inside = (f < grid[0]) & (i < grid[1]) & (j < grid[2])
    token = (f * grid[1] + i) * grid[2] + j
    shape = (_volume(n), _volume(block))
    return torch.where(inside, token, 0).reshape(shape), inside.reshape(shape)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = {"select": _prepare_blocks, "blocks": _prepare_blocks, "append": _prepare_append, "paged": _prepare_paged}
    state = kind[case["op"]](case, g)
    state["case"] = case
    return state


def _normal(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(torch.bfloat16)


def _smooth(rows, B, D, g):
    """Rows that vary slowly along the sequence, as the keys and queries of neighbouring video tokens do."""
    step = 40
    coarse = torch.randn((B, -(-rows // step), D), generator=g, device="cuda")
    x = torch.randn((B, rows, D), generator=g, device="cuda")
    x += 0.7 * coarse.repeat_interleave(step, 1)[:, :rows]
    return (x * 0.82).to(torch.bfloat16)


def _prepare_blocks(case, g):
    B, D = case["B"], case["heads"] * HD
    qg, kg, qb, kb = (_grid(case, key) for key in ("qg", "kg", "qb", "kb"))
    nq, nk, topk = _count(qg, qb), _count(kg, kb), case["topk"]
    Lq, Lk = _volume(qg), _volume(kg)
    if qg == kg:  # column slices of one packed q, k, v projection
        qkv = torch.empty((B, Lk, 3 * D), dtype=torch.bfloat16, device="cuda")
        for n in range(3):
            qkv[:, :, n * D:(n + 1) * D] = _smooth(Lk, B, D, g) if n < 2 else _normal((B, Lk, D), g)
        q, k, v = qkv[:, :, :D], qkv[:, :, D:2 * D], qkv[:, :, 2 * D:]
    else:
        q, k, v = _smooth(Lq, B, D, g), _smooth(Lk, B, D, g), _normal((B, Lk, D), g)
    state = {"q": q, "k": k, "v": v}
    if case["op"] == "select":
        state["mask"] = None
        if case["masked"]:  # the first blocks always, of frames more than eight away none
            fq = torch.arange(nq, device="cuda") // (nq // _numbers(qg, qb)[0]) * qb[0]
            fk = torch.arange(nk, device="cuda") // (nk // _numbers(kg, kb)[0]) * kb[0]
            near = (fq[:, None] - fk[None, :]).abs() <= 8
            always = torch.arange(nk, device="cuda") < topk // 4
            state["mask"] = torch.where(always[None, :], 2, near.to(torch.int32)).to(torch.uint8)
        return state
    chance = torch.rand((B, case["heads"], nq, nk), generator=g, device="cuda")
    picked = chance.topk(topk, -1).indices.sort(-1).values.to(torch.int32)
    counts = torch.full((B, case["heads"], nq), topk, dtype=torch.int32, device="cuda")
    if case["ragged"]:
        counts = torch.randint(0, topk + 1, counts.shape, generator=g, device="cuda", dtype=torch.int32)
    keep = torch.arange(topk, device="cuda") < counts[..., None]
    state["blocks"], state["counts"] = torch.where(keep, picked, -1), counts
    return state


def _pages(B, per, g):
    """A page table whose pages lie in no order, and a few pages that nobody owns."""
    total = B * per + 3
    order = torch.randperm(total, generator=g, device="cuda")[:B * per]
    return order.view(B, per).to(torch.int32), total


def _prepare_append(case, g):
    B, T, D, page = case["B"], case["T"], case["heads"] * HD, case["page"]
    room = max(case["frames"] * case["H"] * case["W"], T)
    table, total = _pages(B, -(-room // page), g)
    state = {"table": table}
    state["k_cache"] = torch.zeros((total, page, D), dtype=torch.bfloat16, device="cuda")
    state["v_cache"] = torch.zeros((total, page, D), dtype=torch.bfloat16, device="cuda")
    qkv = _normal((B, T, 3 * D), g)
    state["q"], state["k"], state["v"] = qkv[:, :, :D], qkv[:, :, D:2 * D], qkv[:, :, 2 * D:]
    count = torch.full((B,), T, dtype=torch.int32, device="cuda")
    start = torch.full((B,), room - T, dtype=torch.int32, device="cuda")
    if case["ragged"]:
        count = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        count[0] = T
        start = (torch.rand((B,), generator=g, device="cuda") * (room - T + 1)).to(torch.int32).clamp(max=room - T)
    state["start"], state["count"] = start, count
    state["q_gain"] = state["k_gain"] = None
    if case["norm"]:
        state["q_gain"] = 1 + 0.1 * torch.randn((D,), generator=g, device="cuda")
        state["k_gain"] = 1 + 0.1 * torch.randn((D,), generator=g, device="cuda")
    return state


def _prepare_paged(case, g):
    B, T, D, page, length = case["B"], case["T"], case["heads"] * HD, case["page"], case["length"]
    table, total = _pages(B, -(-length // page), g)
    lens = torch.full((B,), length, dtype=torch.int32, device="cuda")
    if case["ragged"]:
        lens = (torch.rand((B,), generator=g, device="cuda") * (length + 1)).to(torch.int32).clamp(max=length)
        lens[-1] = length
    k_cache, v_cache = _normal((total, page, D), g), _normal((total, page, D), g)
    return {"q": _normal((B, T, D), g), "k_cache": k_cache, "v_cache": v_cache, "table": table, "lens": lens}


# ---------------------------------------------------------------- the operators
def run(state):
    case = state["case"]
    kind = {"select": _run_select, "blocks": _run_blocks, "append": _run_append, "paged": _run_paged}
    return kind[case["op"]](state, case)


def _run_select(s, c):
    qg, kg, qb, kb = (_grid(c, key) for key in ("qg", "kg", "qb", "kb"))
    if own:
        from video_diffusion_transformer_dit_b200 import binding
        blocks, counts = binding.op_block_select(s["q"], s["k"], c["heads"], qg, kg, qb, kb, c["topk"], mask=s["mask"])
        return {"blocks": blocks, "counts": counts}
    score = _pooled(s["q"], c["heads"], qg, qb) @ _pooled(s["k"], c["heads"], kg, kb).transpose(-1, -2)
    score = torch.where(score.isnan(), -math.inf, score)
    nk, topk = score.shape[-1], c["topk"]
    mask = torch.ones((1, nk), dtype=torch.uint8, device=score.device) if s["mask"] is None else s["mask"]
    mask = mask.expand(score.shape)
    score = torch.where(mask == 2, math.inf, score)
    by_score = score.sort(dim=-1, descending=True, stable=True).indices
    by_mask = mask.gather(-1, by_score).sort(dim=-1, descending=True, stable=True)
    chosen = by_score.gather(-1, by_mask.indices)[..., :topk]
    valid = by_mask.values[..., :topk] > 0
    blocks = torch.where(valid, chosen, nk).sort(-1).values
    blocks = torch.where(blocks < nk, blocks, -1).to(torch.int32)
    return {"blocks": blocks, "counts": valid.sum(-1).to(torch.int32)}


def _pooled(x, heads, grid, block):
    """Mean of each block's tokens inside the grid, in 64 bits: scores next to the border decide the choice."""
    B, n = x.shape[0], _numbers(grid, block)
    x = x.reshape(B, *grid, heads * HD).double()
    x = torch.nn.functional.pad(x, (0, 0) + sum(((0, n[a] * block[a] - grid[a]) for a in (2, 1, 0)), ()))
    x = x.view(B, n[0], block[0], n[1], block[1], n[2], block[2], heads, HD).sum((2, 4, 6))
    _, inside = _tokens(grid, block, x.device)
    x = x.view(B, _volume(n), heads, HD) / inside.sum(-1).double()[None, :, None, None]
    return x.transpose(1, 2)


def _softmax_rows(score, keep, v):
    """softmax(score) v over the kept keys and the logarithm of its sum; rows with none: zero and -inf."""
    score = torch.where(keep, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0, 1.0, total)
    return out, (top + total.log()).squeeze(-1)


def _run_blocks(s, c):
    qg, kg, qb, kb = (_grid(c, key) for key in ("qg", "kg", "qb", "kb"))
    B, heads = c["B"], c["heads"]
    if own:
        from video_diffusion_transformer_dit_b200 import binding
        lse = torch.empty((B, heads, _volume(qg)), dtype=torch.float32, device=s["q"].device)
        out = binding.op_attention_blocks(s["q"], s["k"], s["v"], heads, qg, kg, qb, kb, s["blocks"], s["counts"], lse=lse)
        return {"out": out, "lse": lse}
    dev = s["q"].device
    Lq, Lk, nq = _volume(qg), _volume(kg), _count(qg, qb)
    tq, inq = _tokens(qg, qb, dev)
    tk, ink = _tokens(kg, kb, dev)
    q = s["q"].reshape(B, Lq, heads, HD)[:, tq].float().permute(0, 3, 1, 2, 4)            # [B, h, nq, qv, d]
    at = s["blocks"].clamp(min=0).long()
    used = torch.arange(c["topk"], device=dev) < s["counts"][..., None]
    keys = tk[at].reshape(B, heads, nq, -1)                                               # [B, h, nq, topk kv]
    keep = (ink[at] & used[..., None]).reshape(B, heads, nq, 1, -1)
    b = torch.arange(B, device=dev).view(B, 1, 1, 1)
    h = torch.arange(heads, device=dev).view(1, heads, 1, 1)
    k = s["k"].reshape(B, Lk, heads, HD)[b, keys, h].float()
    score = (q @ k.transpose(-1, -2)) / math.sqrt(HD)
    del k
    v = s["v"].reshape(B, Lk, heads, HD)[b, keys, h].float()
    o, lse = _softmax_rows(score, keep, v)
    place = torch.zeros(Lq, dtype=torch.long, device=dev)                                 # where a token's row is
    row = torch.where(inq, torch.arange(tq.numel(), device=dev).view(tq.shape), 0)
    place = place.scatter_add(0, tq.reshape(-1), row.reshape(-1))
    o = o.reshape(B, heads, -1, HD)[:, :, place].permute(0, 2, 1, 3).reshape(B, Lq, heads * HD)
    return {"out": o.to(torch.bfloat16), "lse": lse.reshape(B, heads, -1)[:, :, place]}


def _turn(x, position, H, W):
    """The three-axis rotation of x [B, T, heads, 128] at cache slots `position` [B, T]; angles in 64 bits."""
    angles = []
    for width, at in ((44, position // (H * W)), (42, position // W % H), (42, position % W)):
        freq = THETA ** (-torch.arange(0, width, 2, dtype=torch.float64, device=x.device) / width)
        angles.append(at.double()[..., None] * freq)
    angle = torch.cat(angles, -1)
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    x = x.unflatten(-1, (HD // 2, 2))
    return torch.stack((x[..., 0] * cos - x[..., 1] * sin, x[..., 0] * sin + x[..., 1] * cos), -1).flatten(-2)


def _run_append(s, c):
    B, T, heads, page = c["B"], c["T"], c["heads"], c["page"]
    if own:
        from video_diffusion_transformer_dit_b200 import binding
        q = binding.op_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["start"], heads, (c["H"], c["W"]),
                                 count=s["count"] if c["ragged"] else None, k_gain=s["k_gain"], q=s["q"],
                                 q_gain=s["q_gain"], eps=EPS)
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "q": q}
    t = torch.arange(T, device=s["k"].device)
    slot = s["start"].long()[:, None] + t
    valid = (t < s["count"][:, None]).reshape(-1)

    def rotated(x, gain):
        x = x.float()
        if gain is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain
        return _turn(x.reshape(B, T, heads, HD), slot, c["H"], c["W"]).reshape(B, T, heads * HD).to(torch.bfloat16)

    to = (s["table"].long().gather(1, slot // page) * page + slot % page).reshape(-1)
    first = valid.to(torch.uint8).argmax()  # its row again in the place of rows that are not appended
    row = torch.where(valid, torch.arange(B * T, device=valid.device), first)
    D = heads * HD
    s["k_cache"].view(-1, D).index_copy_(0, to[row], rotated(s["k"], s["k_gain"]).reshape(-1, D)[row])
    s["v_cache"].view(-1, D).index_copy_(0, to[row], s["v"].reshape(-1, D)[row])
    q = torch.where(valid.view(B, T, 1), rotated(s["q"], s["q_gain"]), 0)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "q": q}


def _run_paged(s, c):
    B, T, heads, page, length = c["B"], c["T"], c["heads"], c["page"], c["length"]
    if own:
        from video_diffusion_transformer_dit_b200 import binding
        lse = torch.empty((B, heads, T), dtype=torch.float32, device=s["q"].device)
        out = binding.op_attention_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], heads, lse=lse)
        return {"out": out, "lse": lse}
    slot = torch.arange(length, device=s["q"].device)
    at = s["table"].long()[:, slot // page] * page + slot % page                          # [B, length]
    keep = (slot < s["lens"][:, None])[:, None, None]
    q = s["q"].reshape(B, T, heads, HD).float().transpose(1, 2)
    k = s["k_cache"].view(-1, heads, HD)[at].float().transpose(1, 2)
    score = (q @ k.transpose(-1, -2)) / math.sqrt(HD)
    del k
    v = s["v_cache"].view(-1, heads, HD)[at].float().transpose(1, 2)
    o, lse = _softmax_rows(score, keep, v)
    return {"out": o.transpose(1, 2).reshape(B, T, heads * HD).to(torch.bfloat16), "lse": lse}


# ---------------------------------------------------------------- work
def work(case):
    B, D, op = case["B"], case["heads"] * HD, case["op"]
    if op in ("select", "blocks"):
        qg, kg, qb, kb = (_grid(case, key) for key in ("qg", "kg", "qb", "kb"))
        Lq, Lk, nq, nk = _volume(qg), _volume(kg), _count(qg, qb), _count(kg, kb)
        lists = B * case["heads"] * nq * (case["topk"] + 1) * 4
        if op == "select":
            return {"bytes": 2 * B * D * (Lq + Lk) + lists + (nq * nk if case["masked"] else 0),
                    "flops": B * D * (Lq + Lk) + 2 * B * D * nq * nk}
        # keys that one list holds: whole blocks of an even share of the tokens
        held = case["topk"] * Lk / nk * (0.5 if case["ragged"] else 1.0)
        return {"bytes": 2 * B * D * (2 * Lq + min(1.0, held * nq / Lk) * 2 * Lk) + lists + 4 * B * case["heads"] * Lq,
                "flops": 4 * B * D * Lq * held}
    if op == "append":
        rows = B * case["T"] * (0.5 if case["ragged"] else 1.0)
        return {"bytes": rows * D * 2 * 6, "flops": rows * D * (20 if case["norm"] else 12)}
    keys = B * case["length"] * (0.5 if case["ragged"] else 1.0)
    return {"bytes": 2 * D * (2 * keys + 2 * B * case["T"]) + 4 * B * case["heads"] * case["T"], "flops": 4 * D * keys * case["T"]}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    kind = {"select": _exact_select, "blocks": _exact_blocks, "append": _exact_append, "paged": _exact_paged}
    return kind[case["op"]](s, case)


def _exact_select(s, c):
    return None  # numbers of blocks and their counts: whole numbers


def _attend(q, k, v):
    """One head: q [n, 128] over k, v [m, 128], all in 64 bits."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    logits = q @ k.T / HD ** 0.5
    return torch.softmax(logits, -1) @ v, torch.logsumexp(logits, -1)


def _block_of(grid, block, device):
    """The block that each token lies in."""
    n = _numbers(grid, block)
    f, i, j = torch.meshgrid(*(torch.arange(g, device=device) for g in grid), indexing="ij")
    return (((f // block[0]) * n[1] + i // block[1]) * n[2] + j // block[2]).reshape(-1)


def _exact_blocks(s, c):
    qg, kg, qb, kb = (_grid(c, key) for key in ("qg", "kg", "qb", "kb"))
    B, heads, Lq, dev = c["B"], c["heads"], _volume(qg), s["q"].device
    nk = _count(kg, kb)
    mine, theirs = _block_of(qg, qb, dev), _block_of(kg, kb, dev)
    out = torch.zeros((B, Lq, heads * HD), dtype=torch.float64, device=dev)
    lse = torch.zeros((B, heads, Lq), dtype=torch.float64, device=dev)
    for b in range(B):
        for h in range(heads):
            part = slice(h * HD, (h + 1) * HD)
            q, k, v = (s[n][b, :, part].double() for n in ("q", "k", "v"))
            listed_, count = s["blocks"][b, h].long(), s["counts"][b, h].long()
            allowed = torch.zeros((listed_.shape[0], nk + 1), dtype=torch.bool, device=dev)
            there = torch.arange(listed_.shape[1], device=dev) < count[:, None]
            allowed.scatter_(1, torch.where(there, listed_, nk), True)
            for rows in torch.arange(Lq, device=dev).split(4096):
                sees = allowed[mine[rows]][:, theirs]
                logits = (q[rows] @ k.T / HD ** 0.5).masked_fill(~sees, -math.inf)
                lse[b, h, rows] = torch.logsumexp(logits, -1)
                out[b, rows, part] = torch.softmax(logits, -1).nan_to_num(0.0) @ v
    return {"out": out, "lse": lse}


def _exact_append(s, c):
    B, T, heads, page, H, W = (c[n] for n in ("B", "T", "heads", "page", "H", "W"))
    dev, D = s["k"].device, heads * HD
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    q_out = torch.zeros((B, T, D), dtype=torch.float64, device=dev)
    widths = (44, 42, 42)
    pair = torch.cat([torch.arange(w // 2, dtype=torch.float64, device=dev) * 2 / w for w in widths])
    rate = torch.exp(-math.log(THETA) * pair)
    for b in range(B):
        n, first = int(s["count"][b]), int(s["start"][b])
        slot = first + torch.arange(n, device=dev)
        place = torch.stack((slot // (H * W), slot % (H * W) // W, slot % W)).double()
        axis = torch.repeat_interleave(torch.tensor([0, 1, 2], device=dev), torch.tensor([w // 2 for w in widths], device=dev))
        unit = torch.polar(torch.ones((), dtype=torch.float64, device=dev), place[axis].T * rate)
        for name, gain in (("k", s["k_gain"]), ("q", s["q_gain"])):
            x = s[name][b, :n].double()
            if gain is not None:
                x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * gain.double()
            turned = torch.view_as_real(torch.view_as_complex(x.reshape(n, heads, HD // 2, 2)) * unit[:, None]).reshape(n, D)
            if name == "q":
                q_out[b, :n] = turned
            else:
                k_cache[s["table"][b].long()[slot // page], slot % page] = turned
        v_cache[s["table"][b].long()[slot // page], slot % page] = s["v"][b, :n].double()
    return {"k_cache": k_cache, "v_cache": v_cache, "q": q_out}


def _exact_paged(s, c):
    B, T, heads, page, dev = c["B"], c["T"], c["heads"], c["page"], s["q"].device
    out = torch.zeros((B, T, heads * HD), dtype=torch.float64, device=dev)
    lse = torch.zeros((B, heads, T), dtype=torch.float64, device=dev)
    for b in range(B):
        n = int(s["lens"][b])
        mine = s["table"][b, :-(-n // page)].long()
        for h in range(heads):
            part = slice(h * HD, (h + 1) * HD)
            k, v = (s[name][mine][:, :, part].reshape(-1, HD)[:n].double() for name in ("k_cache", "v_cache"))
            out[b, :, part], lse[b, h] = _attend(s["q"][b, :, part].double(), k, v)
    return {"out": out, "lse": lse}
