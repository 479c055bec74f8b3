"""Definitions in 64 bits of the attention operators over parts of the sequence, for their tests."""
import math

import torch

HD = 128
HALF_STEP = 2.0 ** -8          # bf16 rounding: half a step relative to the value
DT = torch.float64


def numbers(grid, block):
    return [-(-g // b) for g, b in zip(grid, block)]


def volume(d):
    return d[0] * d[1] * d[2]


def block_count(grid, block):
    return volume(numbers(grid, block))


def block_of(grid, block, device="cpu"):
    """Block of each token, in token order."""
    n = numbers(grid, block)
    f, i, j = torch.meshgrid(*(torch.arange(g, device=device) for g in grid), indexing="ij")
    return (((f // block[0]) * n[1] + i // block[1]) * n[2] + j // block[2]).reshape(-1)


def select(q, k, heads, qg, kg, qb, kb, topk, mask=None):
    """(blocks, counts) by sorting (rank of the mask, score, block) row by row."""
    B = q.shape[0]
    nq, nk = block_count(qg, qb), block_count(kg, kb)
    mine, theirs = block_of(qg, qb), block_of(kg, kb)
    blocks = torch.full((B, heads, nq, topk), -1, dtype=torch.int32)
    counts = torch.zeros((B, heads, nq), dtype=torch.int32)

    def means(x, of, n):
        x = x.cpu().to(DT).reshape(B, -1, heads, HD)
        out = torch.zeros(B, n, heads, HD, dtype=DT).index_add_(1, of, x)
        return out / torch.bincount(of, minlength=n).to(DT)[None, :, None, None]

    score = torch.einsum("bihd,bjhd->bhij", means(q, mine, nq), means(k, theirs, nk)).tolist()
    kind = torch.ones(nq, nk).tolist() if mask is None else mask.cpu().clamp(max=2).tolist()
    for b in range(B):
        for h in range(heads):
            for i in range(nq):
                row = [(-kind[i][j], 0.0 if kind[i][j] == 2 else (math.inf if math.isnan(s) else -s), j)
                       for j, s in enumerate(score[b][h][i]) if kind[i][j] > 0]
                keep = sorted(j for _, _, j in sorted(row)[:topk])
                blocks[b, h, i, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
                counts[b, h, i] = len(keep)
    return blocks, counts


def attend(q, k, v, weight):
    """softmax(q k^T / sqrt(128)) v of one head with whole-number key weights [n, m] (0: not there, 2: listed
    twice): output, log of the denominator, sum of p |v| (what the rounding of p can move) and the largest sum
    of |q| |k| (what the fp32 sums of the logits can move)."""
    logits = q @ k.T / HD ** 0.5
    logits = torch.where(weight > 0, logits, -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.where(weight > 0, weight * (logits - top).exp(), 0.0)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    size = torch.where(weight > 0, (q.abs() @ k.abs().T) / HD ** 0.5, 0.0).amax(-1)
    return p @ v, (top + total.log()).squeeze(-1), p @ v.abs(), size


def check_attention(out, lse, ref, ref_lse, moved, size):
    """out (bf16) and lse against the 64-bit values.  Each p is rounded to bf16 once (2^-8 of it) and the output
    once (2^-8); a logit is a sum of 128 exact products in fp32 (at most 128 roundings of 2^-24 of the sum of
    their sizes, and the scale's), and moves every p by as much; exp2 and the sums add a few 2^-22."""
    logit = (130 * 2.0 ** -24) * size
    bound = HALF_STEP * 1.01 * (moved + ref.abs()) + (2 * logit[..., None] + 2.0 ** -18) * moved + 1e-30
    off = (out.to(DT) - ref).abs()
    assert bool((off <= bound).all()), f"largest excess {(off - bound).max().item():.3g}"
    if lse is not None:
        none = ref_lse == -math.inf
        assert torch.equal(lse.to(DT) == -math.inf, none)
        off = torch.where(none, 0.0, (lse.to(DT) - ref_lse).abs())
        far = off - (logit + 2.0 ** -18 + 2.0 ** -22 * ref_lse.abs().nan_to_num(0, 0, 0))
        assert bool((far <= 0).all()), f"lse: largest excess {far.max().item():.3g}"


def attention_blocks(q, k, v, heads, qg, kg, qb, kb, blocks, counts):
    B, dev = q.shape[0], q.device
    Lq, nk = volume(qg), block_count(kg, kb)
    mine, theirs = block_of(qg, qb, dev), block_of(kg, kb, dev)
    o, moved = (torch.zeros(B, Lq, heads * HD, dtype=DT, device=dev) for _ in range(2))
    lse, size = (torch.zeros(B, heads, Lq, dtype=DT, device=dev) for _ in range(2))
    there = torch.arange(blocks.shape[-1], device=dev) < counts[..., None]
    there &= (blocks >= 0) & (blocks < nk)
    for b in range(B):
        for h in range(heads):
            part = slice(h * HD, (h + 1) * HD)
            weight = torch.zeros(blocks.shape[2], nk + 1, dtype=DT, device=dev)
            at = torch.where(there[b, h], blocks[b, h], nk).long()
            weight.scatter_add_(1, at, torch.ones_like(at, dtype=DT))
            o[b, :, part], lse[b, h], moved[b, :, part], size[b, h] = attend(
                q[b, :, part].to(DT), k[b, :, part].to(DT).nan_to_num(0, 0, 0), v[b, :, part].to(DT).nan_to_num(0, 0, 0),
                weight[mine][:, theirs])
    return o, lse, moved, size.transpose(1, 2).repeat_interleave(HD, -1)


def gathered(cache, table, n):
    """The first n places of a sequence, and whether each is in a page that is there."""
    page = cache.shape[1]
    slot = torch.arange(n, device=cache.device)
    at = table.long()[slot // page]
    ok = (at >= 0) & (at < cache.shape[0])
    return torch.where(ok[:, None], cache[at.clamp(0, cache.shape[0] - 1), slot % page].to(DT), 0.0), ok


def attention_paged(q, k_cache, v_cache, table, lens, heads):
    B, T, dev = q.shape[0], q.shape[1], q.device
    o, moved = (torch.zeros(B, T, heads * HD, dtype=DT, device=dev) for _ in range(2))
    lse, size = (torch.zeros(B, heads, T, dtype=DT, device=dev) for _ in range(2))
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * k_cache.shape[1])
        k, ok = gathered(k_cache, table[b], n)
        v, _ = gathered(v_cache, table[b], n)
        for h in range(heads):
            part = slice(h * HD, (h + 1) * HD)
            if n == 0:
                lse[b, h] = -math.inf
                continue
            o[b, :, part], lse[b, h], moved[b, :, part], size[b, h] = attend(
                q[b, :, part].to(DT), k[:, part], v[:, part], ok.to(DT).expand(T, n))
    return o, lse, moved, size.transpose(1, 2).repeat_interleave(HD, -1)


def rotated(x, slot, heads, hw, gain, eps=1e-6, split=(44, 42, 42), theta=10000.0, rope=True):
    """x [T, D] (64 bits) normed across heads and turned at the places `slot`; and the size of what each output
    sums up (|a| + |b| of its pair)."""
    if gain is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * gain.to(DT)
    x = x.reshape(-1, heads, HD // 2, 2)
    size = x.abs().sum(-1, keepdim=True).expand_as(x).reshape(-1, heads * HD)
    if rope:
        H, W = hw
        place = torch.stack((slot // (H * W), slot // W % H, slot % W)).to(DT)
        angle = torch.cat([place[a][:, None] * theta ** (-torch.arange(0, w, 2, dtype=DT, device=x.device) / w)
                           for a, w in enumerate(split)], -1)
        x = torch.view_as_real(torch.view_as_complex(x.contiguous()) * torch.polar(torch.ones_like(angle), angle)[:, None])
    return x.reshape(-1, heads * HD), size


def block_means(x, heads, grid, block):
    """Mean of each block [B, heads, blocks, 128] in 64 bits, its tokens added one after the other in token order."""
    of, n = block_of(grid, block, x.device), block_count(grid, block)
    order = of.argsort(stable=True)
    count = torch.bincount(of, minlength=n)
    place = torch.arange(of.numel(), device=x.device) - (count.cumsum(0) - count)[of[order]]
    token = torch.full((n, volume(block)), of.numel(), device=x.device)
    token[of[order], place] = order
    x = torch.cat((x, torch.zeros_like(x[:, :1])), 1)
    total = torch.zeros(x.shape[0], n, x.shape[2], dtype=DT, device=x.device)
    for t in range(volume(block)):
        total += torch.where((token[:, t] < of.numel())[:, None], x[:, token[:, t]].to(DT), 0.0)
    return (total / count.to(DT)[:, None]).view(x.shape[0], n, heads, HD).transpose(1, 2)


def select_rows(q, k, heads, qg, kg, qb, kb, topk, mask=None):
    """What select() gives, by sorting all rows at once on the tensors' device."""
    score = block_means(q, heads, qg, qb) @ block_means(k, heads, kg, kb).transpose(-1, -2)
    nk = score.shape[-1]
    kind = torch.ones(score.shape[-2:], dtype=torch.long) if mask is None else mask.cpu().clamp(max=2).long()
    kind = kind.to(score.device).expand(score.shape)
    score = torch.where(kind == 2, 0.0, torch.where(score.isnan(), -math.inf, score))
    rank = score.argsort(dim=-1, descending=True, stable=True)
    rank = rank.gather(-1, kind.gather(-1, rank).argsort(dim=-1, descending=True, stable=True))[..., :topk]
    keep = torch.where(kind.gather(-1, rank) > 0, rank, nk).sort(-1).values
    return torch.where(keep < nk, keep, -1).int().cpu(), (keep < nk).sum(-1).int().cpu()


def check_rows(out, lse, ref, ref_lse, moved, size, keys):
    """As check_attention, for a kernel that keeps p in fp32 (one and two new tokens): the output's rounding (2^-8),
    the logits (130 roundings as there, and two more of the exponent's difference from the row's maximum), 2^-21 of
    exp2 on both sides of the fraction, and the sums: at most keys / 8 additions of a lane one after the other, as
    many rescalings, a few dozen where lanes, warps and parts meet, for numerator and denominator."""
    logit = (132 * 2.0 ** -24) * size
    sums = (keys / 2 + 256) * 2.0 ** -24 + 2.0 ** -20
    bound = HALF_STEP * 1.01 * ref.abs() + (2 * logit[..., None] + sums) * moved + 1e-30
    off = (out.to(DT) - ref).abs()
    assert bool((off <= bound).all()), f"largest excess {(off - bound).max().item():.3g}"
    if lse is not None:
        none = ref_lse == -math.inf
        assert torch.equal(lse.to(DT) == -math.inf, none)
        off = torch.where(none, 0.0, (lse.to(DT) - ref_lse).abs())
        far = off - (logit + sums + 2.0 ** -22 * ref_lse.abs().nan_to_num(0, 0, 0))
        assert bool((far <= 0).all()), f"lse: largest excess {far.max().item():.3g}"


# q . k / sqrt(128) in log2 units is -b for marked_query() and keys whose first two columns hold -b: bf16's 7.84375
# and what is left of sqrt(128) / log2(e) (to 4e-7 of it), so p is a power of two and its rounding to bf16 exact.
def marked_query(shape, device):
    q = torch.zeros(shape, dtype=torch.bfloat16, device=device)
    q[..., 0::HD] = 7.84375
    q[..., 1::HD] = HD ** 0.5 * math.log(2.0) - 7.84375
    return q


def marked_keys(b, heads):
    """Keys [n, heads * 128] of weights 2^-b."""
    k = torch.zeros((*b.shape, heads, HD), dtype=torch.bfloat16, device=b.device)
    k[..., :2] = -b[..., None, None].to(torch.bfloat16)
    return k.flatten(-2)


def marked_values(n, first, heads, device):
    """Values [n, heads * 128]: of keys first .. first + 127 a one in a column of its own, else zero."""
    v = torch.zeros((n, heads, HD), dtype=torch.bfloat16, device=device)
    at = torch.arange(first, min(first + HD, n), device=device)
    v[at, :, at - first] = 1
    return v.flatten(-2)


def check_marked(out, weight, first):
    """out [..., heads, 128] where the keys have these weights [..., 1 or heads, n] of a row: each column is one key's.
    The output's rounding, 4e-7 * b of the weights and the sums."""
    total = weight.sum(-1, keepdim=True)
    want = (weight / torch.where(total == 0, 1.0, total))[..., first:first + HD]
    got = out[..., :want.shape[-1]].to(DT)
    off = (got - want).abs()
    assert bool((off <= want * (HALF_STEP * 1.01 + 2.0 ** -14)).all()), f"{(off / want.clamp(min=1e-30)).max().item():.3g}"
    assert bool((out[..., want.shape[-1]:] == 0).all())
