"""Attention over parts of the sequence on the GPU: block selection, block-sparse attention, appending to a
paged cache and attention over it, against their definitions in 64 bits."""
import math

import pytest
import torch

from tests import attention_parts as R
from tests.gpu_common import DT, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    from video_diffusion_transformer_dit_b200 import binding
    binding.lib()


def B():
    from video_diffusion_transformer_dit_b200 import binding
    return binding


def rnd(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def packed(Bn, L, heads, seed):
    qkv = rnd((Bn, L, 3 * heads * 128), seed)
    return qkv.split(heads * 128, -1)


# ------------------------------------------------------------------ selection
SELECT = [  # B, heads, q grid, k grid, q block, k block, topk
    (1, 1, (1, 1, 1), (1, 1, 1), (1, 1, 1), (1, 1, 16), 1),
    (2, 3, (3, 8, 8), (3, 8, 8), (1, 8, 8), (1, 4, 4), 5),
    (1, 2, (5, 7, 11), (5, 7, 11), (3, 5, 7), (4, 4, 4), 4),
    (1, 2, (2, 5, 9), (7, 9, 20), (4, 4, 8), (2, 4, 4), 11),
    (1, 1, (1, 1, 333), (1, 1, 9000), (1, 1, 128), (1, 1, 16), 60),     # 563 key blocks
    (1, 1, (1, 1, 300), (1, 1, 20001), (1, 1, 64), (1, 1, 16), 100),    # 1251 key blocks
    (1, 17, (2, 8, 8), (2, 8, 8), (1, 8, 16), (1, 8, 8), 2),
]


@pytest.mark.parametrize("case", SELECT)
def test_block_select(case):
    Bn, heads, qg, kg, qb, kb, topk = case
    q, k = rnd((Bn, R.volume(qg), heads * 128), 1), rnd((Bn, R.volume(kg), heads * 128), 2)
    blocks, counts = B().op_block_select(q, k, heads, qg, kg, qb, kb, topk)
    B().op_sync()
    want = R.select(q, k, heads, qg, kg, qb, kb, topk)
    assert torch.equal(blocks.cpu(), want[0]) and torch.equal(counts.cpu(), want[1])


@pytest.mark.parametrize("nk", [100, 500, 1000, 1300])
def test_block_select_masks_leave_rows_empty_short_and_full(nk):
    heads, topk = 2, 7
    qg, kg, qb, kb = (1, 1, 6 * 32), (1, 1, nk * 16 - 3), (1, 1, 32), (1, 1, 16)
    q, k = rnd((1, qg[2], heads * 128), 3), rnd((1, kg[2], heads * 128), 4)
    mask = torch.ones(6, nk, dtype=torch.uint8)
    mask[0] = 0                                  # nothing
    mask[1] = 0
    mask[1, [nk - 1, 3, 17]] = 1                 # fewer than topk
    mask[2, :20] = 2                             # more asked for than topk: the lowest blocks
    mask[3, nk - 3:] = 2                         # some asked for, the rest by score
    mask[4, ::2] = 0
    blocks, counts = B().op_block_select(q, k, heads, qg, kg, qb, kb, topk, mask=mask.cuda())
    B().op_sync()
    want = R.select(q, k, heads, qg, kg, qb, kb, topk, mask)
    assert torch.equal(blocks.cpu(), want[0]) and torch.equal(counts.cpu(), want[1])
    assert counts[0, 0].tolist() == [0, 3, 7, 7, 7, 7]


@pytest.mark.parametrize("nk", [64, 700, 1500])
def test_block_select_equal_scores_go_to_the_lowest_blocks(nk):
    heads, topk = 1, 30
    kb, kg = (1, 1, 16), (1, 1, nk * 16)
    pattern = rnd((5, 16, 128), 5)
    k = pattern[torch.arange(nk, device="cuda") % 5].reshape(1, nk * 16, 128).contiguous()
    q = rnd((1, 40, 128), 6)
    q[0, 32:] = 0                                # a block of zero queries: every score is 0
    args = (heads, (1, 1, 40), kg, (1, 1, 32), kb, topk)
    blocks, counts = B().op_block_select(q, k, *args)
    B().op_sync()
    want = R.select(q, k, *args)
    assert torch.equal(blocks.cpu(), want[0]) and torch.equal(counts.cpu(), want[1])
    assert blocks[0, 0, 1].tolist() == list(range(30))


@pytest.mark.parametrize("nk", [40, 1100])
def test_block_select_ranks_nan_and_infinite_scores(nk):
    kg = (1, 1, nk * 16)
    q, k = rnd((1, 16, 128), 7).abs(), rnd((1, nk * 16, 128), 8)
    k[0, 5 * 16 + 2, 7] = math.nan               # ranks with -inf
    k[0, 9 * 16, 0] = math.inf                   # first
    k[0, 11 * 16, 0] = -math.inf
    for topk in (1, nk - 1, nk):
        blocks, counts = B().op_block_select(q, k, 1, (1, 1, 16), kg, (1, 1, 16), (1, 1, 16), topk)
        B().op_sync()
        want = R.select(q, k, 1, (1, 1, 16), kg, (1, 1, 16), (1, 1, 16), topk)
        assert torch.equal(blocks.cpu(), want[0]) and int(counts) == topk


# ------------------------------------------------------------------ block-sparse attention
def lists(Bn, heads, nq, nk, topk, seed, ragged=True):
    g = torch.Generator().manual_seed(seed)
    blocks = torch.rand((Bn, heads, nq, nk), generator=g).topk(topk, -1).indices.sort(-1).values.to(torch.int32)
    counts = torch.full((Bn, heads, nq), topk, dtype=torch.int32)
    if ragged:
        counts = torch.randint(0, topk + 1, counts.shape, generator=g, dtype=torch.int32)
    return blocks.cuda(), counts.cuda()


BLOCKS = [  # B, heads, q grid, k grid, q block, k block, topk, ragged
    (1, 1, (1, 1, 1), (1, 1, 1), (1, 1, 1), (1, 1, 16), 1, False),
    (1, 1, (1, 1, 1), (1, 1, 700), (1, 1, 128), (1, 1, 64), 11, False),        # one token, split list
    (2, 3, (3, 8, 8), (3, 8, 8), (1, 8, 8), (1, 4, 4), 6, True),
    (1, 2, (5, 7, 11), (5, 7, 11), (3, 5, 7), (4, 4, 4), 8, True),             # 105-token query blocks, ragged edges
    (1, 2, (1, 9, 13), (7, 9, 13), (1, 8, 16), (2, 8, 8), 6, False),           # frame on window, split
    (2, 2, (5, 9, 9), (5, 9, 9), (4, 4, 8), (2, 4, 4), 20, True),              # 32-token key blocks
    (1, 40, (6, 8, 8), (6, 8, 8), (1, 4, 8), (1, 8, 8), 3, True),              # 480 units: several per stream
    (1, 2, (1, 1, 2000), (1, 1, 2000), (1, 1, 128), (1, 1, 128), 9, True),
]


@pytest.mark.parametrize("case", BLOCKS)
def test_attention_blocks(case):
    Bn, heads, qg, kg, qb, kb, topk, ragged = case
    if qg == kg:
        q, k, v = packed(Bn, R.volume(qg), heads, 11)
    else:
        q = rnd((Bn, R.volume(qg), heads * 128), 12)
        k, v = rnd((Bn, R.volume(kg), heads * 128), 13), rnd((Bn, R.volume(kg), heads * 128), 14)
    blocks, counts = lists(Bn, heads, R.block_count(qg, qb), R.block_count(kg, kb), topk, 15, ragged)
    lse = torch.full((Bn, heads, R.volume(qg)), math.nan, device="cuda")
    out = B().op_attention_blocks(q, k, v, heads, qg, kg, qb, kb, blocks, counts, lse=lse)
    B().op_sync()
    ref, ref_lse, moved, size = R.attention_blocks(q, k, v, heads, qg, kg, qb, kb, blocks, counts)
    check(out, lse, ref, ref_lse, moved, size)


def check(out, lse, ref, ref_lse, moved, size):
    heads = ref_lse.shape[1]
    Bn, L = out.shape[:2]
    per_head = lambda x: x.reshape(Bn, L, heads, 128).transpose(1, 2)  # noqa: E731
    R.check_attention(per_head(out), lse, per_head(ref), ref_lse, per_head(moved), per_head(size)[..., 0])
    assert bool((out[(ref_lse == -math.inf).transpose(1, 2).repeat_interleave(128, -1)] == 0).all())


@pytest.mark.parametrize("long", [False, True])
def test_attention_blocks_odd_lists_and_foreign_memory(long):
    """Entries outside the grid are skipped, a block listed twice counts twice, counts are held to the list's
    length, and NaN in blocks that are not listed stays out."""
    heads, qg, kg, qb, kb = 2, (2, 4, 8), ((21, 8, 8) if long else (4, 8, 8)), (1, 4, 8), (1, 4, 4)
    nq, nk = R.block_count(qg, qb), R.block_count(kg, kb)
    q, k, v = rnd((1, 64, 256), 21), rnd((1, R.volume(kg), 256), 22), rnd((1, R.volume(kg), 256), 23)
    topk = 20
    blocks, _ = lists(1, heads, nq, nk - 2, min(topk, nk - 2), 24, False)
    if blocks.shape[-1] < topk:
        blocks = torch.cat((blocks, blocks[..., :topk - blocks.shape[-1]]), -1)
    blocks = blocks.contiguous()
    blocks[0, 0, 0, 3] = -1
    blocks[0, 0, 0, 4] = nk
    blocks[0, 0, 1, :] = 2 ** 31 - 1                # nothing left
    blocks[0, 1, 0, 7] = blocks[0, 1, 0, 6]         # twice
    blocks[0, 1, 1, 16:] = -5
    counts = torch.tensor([[[topk, topk], [topk + 9, topk]]], dtype=torch.int32, device="cuda")
    last = R.block_of(kg, kb, "cuda") >= nk - 2     # in no list
    k[0, last] = math.nan
    v[0, last] = math.inf
    lse = torch.empty((1, heads, 64), device="cuda")
    out = B().op_attention_blocks(q, k, v, heads, qg, kg, qb, kb, blocks, counts, lse=lse)
    B().op_sync()
    check(out, lse, *R.attention_blocks(q, k, v, heads, qg, kg, qb, kb, blocks, counts))
    assert bool((lse[0, 0, 32:] == -math.inf).all())


def test_attention_blocks_negative_counts_and_large_logits():
    heads, g, qb, kb = 1, (1, 1, 256), (1, 1, 64), (1, 1, 64)
    q, k, v = rnd((1, 256, 128), 25, 30.0), rnd((1, 256, 128), 26, 30.0), rnd((1, 256, 128), 27)
    blocks = torch.arange(4, dtype=torch.int32, device="cuda").expand(1, 1, 4, 4).contiguous()
    counts = torch.tensor([[[-3, 0, 1, 4]]], dtype=torch.int32, device="cuda")
    lse = torch.empty((1, 1, 256), device="cuda")
    out = B().op_attention_blocks(q, k, v, heads, g, g, qb, kb, blocks, counts, lse=lse)
    B().op_sync()
    assert bool((out[0, :128] == 0).all()) and bool((lse[0, 0, :128] == -math.inf).all())
    check(out, lse, *R.attention_blocks(q, k, v, heads, g, g, qb, kb, blocks, counts))


def test_attention_blocks_infinite_and_nan_inputs_follow_the_formula():
    """-inf logits drop a key, a query whose logits are all -inf gets a zero row, NaN stays in its row."""
    g, b = (1, 1, 64), (1, 1, 64)
    q = torch.zeros((1, 64, 128), dtype=torch.bfloat16, device="cuda")
    q[0, :, 0] = 1
    q[0, 1] = 0
    q[0, 2, 5] = math.nan
    k, v = rnd((1, 64, 128), 28), rnd((1, 64, 128), 29)
    k[0, :32, 0] = -math.inf
    q[0, 1, 1] = 1
    blocks = torch.zeros((1, 1, 1, 1), dtype=torch.int32, device="cuda")
    counts = torch.ones((1, 1, 1), dtype=torch.int32, device="cuda")
    out = B().op_attention_blocks(q, k, v, 1, g, g, b, b, blocks, counts)
    B().op_sync()
    logits = q[0].to(DT) @ k[0].to(DT).T / 128 ** 0.5
    ref = torch.softmax(logits, -1) @ v[0].to(DT)
    assert bool(out[0, 2].isnan().all()) and bool(out[0, 1].isnan().all())   # 0 * -inf is NaN in the formula too
    rows = [0] + list(range(3, 64))
    assert bool(ref[rows].isfinite().all())
    torch.testing.assert_close(out[0, rows].to(DT), ref[rows], rtol=2 * R.HALF_STEP, atol=2 * R.HALF_STEP * 4)
    k[0, :, 0] = -math.inf
    lse = torch.empty((1, 1, 64), device="cuda")
    out = B().op_attention_blocks(q, k, v, 1, g, g, b, b, blocks, counts, lse=lse)
    B().op_sync()
    assert bool((out[0, rows] == 0).all()) and bool((lse[0, 0, rows] == -math.inf).all())


def test_attention_blocks_writes_its_rows_only():
    heads, g, qb, kb = 2, (3, 5, 7), (2, 4, 4), (2, 4, 4)
    L, D = R.volume(g), heads * 128
    q, k, v = packed(2, L, heads, 31)
    nq = R.block_count(g, qb)
    blocks, counts = lists(2, heads, nq, nq, 3, 32)
    wide = torch.full((2 * L + 3, D + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:2 * L].view(2, L, D + 64)[:, :, :D]
    B().op_attention_blocks(q, k, v, heads, g, g, qb, kb, blocks, counts, out=out)
    B().op_sync()
    assert bool((wide[2 * L:] == 7).all()) and bool((wide[:, D:] == 7).all())
    ref, ref_lse, moved, size = R.attention_blocks(q, k, v, heads, g, g, qb, kb, blocks, counts)
    check(out, None, ref, ref_lse, moved, size)


def test_selected_everything_equals_dense_attention_and_a_share_is_near():
    """The pair as it is used: every block kept gives the dense attention; the kept blocks alone are attended."""
    heads, g, qb, kb = 4, (5, 10, 12), (4, 4, 8), (4, 4, 4)
    L = R.volume(g)
    q, k, v = packed(2, L, heads, 33)
    nk = R.block_count(g, kb)
    dense = torch.empty((2 * L, heads * 128), dtype=torch.bfloat16, device="cuda")
    B().op_attention(q, k, v, dense, 2, heads, L, L, ldq=q.stride(1), ldk=k.stride(1), ldv=v.stride(1))
    blocks, counts = B().op_block_select(q, k, heads, g, g, qb, kb, nk)
    assert bool((counts == nk).all())
    out = B().op_attention_blocks(q, k, v, heads, g, g, qb, kb, blocks, counts)
    B().op_sync()
    ref, ref_lse, moved, size = R.attention_blocks(q, k, v, heads, g, g, qb, kb, blocks, counts)
    check(out, None, ref, ref_lse, moved, size)
    check(dense.view(2, L, -1), None, ref, ref_lse, moved, size)
    blocks, counts = B().op_block_select(q, k, heads, g, g, qb, kb, 5)
    out = B().op_attention_blocks(q, k, v, heads, g, g, qb, kb, blocks, counts)
    B().op_sync()
    check(out, None, *R.attention_blocks(q, k, v, heads, g, g, qb, kb, blocks, counts))


# ------------------------------------------------------------------ paged cache
def cache(Bn, per, page, heads, seed, extra=3):
    g = torch.Generator().manual_seed(seed)
    total = Bn * per + extra
    table = torch.randperm(total, generator=g)[:Bn * per].view(Bn, per).to(torch.int32).cuda()
    return rnd((total, page, heads * 128), seed), rnd((total, page, heads * 128), seed + 1), table


APPEND = [  # B, T, heads, (H, W), page, first places, counts, norm
    (1, 1, 1, (1, 1), 16, [0], None, False),
    (3, 5, 2, (2, 3), 16, [0, 14, 31], [5, 0, 3], True),
    (2, 130, 12, (30, 52), 64, [1500, 7], [130, 129], True),
    (2, 9, 40, (4, 4), 128, [120, 250], None, False),
    (1, 20, 3, (5, 7), 32, [70], [99], True),                    # a count above T is T
    (2, 700, 5, (9, 11), 16, [0, 333], [700, 651], True),        # several rows per warp
    (2, 37, 17, (3, 4), 32, [9, 100], None, True),               # two warps per row
    (3, 800, 33, (6, 7), 64, [0, 5, 900], [800, 1, 799], True),  # four
    (1, 70, 96, (5, 5), 16, [3], None, True),                    # eight
]


@pytest.mark.parametrize("case", APPEND)
def test_kv_append(case):
    Bn, T, heads, hw, page, first, count, norm = case
    D = heads * 128
    per = -(-(max(first) + T) // page) + 1
    kc, vc, table = cache(Bn, per, page, heads, 41)
    before = kc.clone(), vc.clone()
    q, k, v = packed(Bn, T, heads, 42)
    qg, kg = (1 + 0.1 * rnd((D,), 43).float(), 1 + 0.1 * rnd((D,), 44).float()) if norm else (None, None)
    start = torch.tensor(first, dtype=torch.int32, device="cuda")
    cnt = None if count is None else torch.tensor(count, dtype=torch.int32, device="cuda")
    q_out = torch.full((Bn, T, D), 5.0, dtype=torch.bfloat16, device="cuda")
    B().op_kv_append(k, v, kc, vc, table, start, heads, hw, count=cnt, k_gain=kg, q=q, q_gain=qg, q_out=q_out)
    B().op_sync()
    want_k, want_v = before
    bound_k = torch.zeros_like(want_k, dtype=DT)
    want_k = want_k.to(DT)
    for b in range(Bn):
        n = min(T if count is None else count[b], T)
        slot = first[b] + torch.arange(n, device="cuda")
        at = table[b].long()[slot // page], slot % page
        y, size = R.rotated(k[b, :n].to(DT), slot, heads, hw, kg)
        want_k[at] = y
        bound_k[at] = R.HALF_STEP * y.abs() * 1.001 + 2.0 ** -20 * size      # one rounding; fp32 sums of two
        want_v[at] = v[b, :n]
        y, size = R.rotated(q[b, :n].to(DT), slot, heads, hw, qg)
        assert bool(((q_out[b, :n].to(DT) - y).abs() <= R.HALF_STEP * 1.001 * y.abs() + 2.0 ** -20 * size).all())
        assert bool((q_out[b, n:] == 5).all())
    assert torch.equal(vc, want_v)
    assert bool(((kc.to(DT) - want_k).abs() <= bound_k).all())


def test_kv_append_far_places_keep_their_angles():
    """Frame numbers of 1e5: the angle keeps its fraction, and the rotation its relative positions."""
    heads, hw, page = 1, (2, 2), 16
    kc, vc, _ = cache(1, 2, page, heads, 45)
    frames = 100003
    place = frames * 4
    table = torch.full((1, place // page + 2), -1, dtype=torch.int32, device="cuda")
    table[0, place // page] = 1
    table[0, place // page + 1] = 0
    q, k, v = packed(1, 6, heads, 46)
    start = torch.tensor([place], dtype=torch.int32, device="cuda")
    q_out = B().op_kv_append(k, v, kc, vc, table, start, heads, hw, q=q)
    B().op_sync()
    slot = place + torch.arange(6, device="cuda")
    y, size = R.rotated(q[0].to(DT), slot, heads, hw, None)
    assert bool(((q_out[0].to(DT) - y).abs() <= R.HALF_STEP * 1.001 * y.abs() + 2.0 ** -20 * size).all())
    got = kc[table[0].long()[slot // page], slot % page].to(DT)
    y, size = R.rotated(k[0].to(DT), slot, heads, hw, None)
    assert bool(((got - y).abs() <= R.HALF_STEP * 1.001 * y.abs() + 2.0 ** -20 * size).all())


def test_kv_append_leaves_places_outside_alone_and_norms_in_place():
    heads, page, T = 2, 16, 40
    kc, vc, table = cache(3, 2, page, heads, 47)
    table[1, 1] = -1
    table[2, 0] = kc.shape[0]
    before = kc.clone(), vc.clone()
    q, k, v = packed(3, T, heads, 48)
    q = q.contiguous()
    was = q.clone()
    start = torch.tensor([20, 0, -1], dtype=torch.int32, device="cuda")     # past the table; a missing page; before it
    got = B().op_kv_append(k, v, kc, vc, table, start, heads, (3, 3), q=q, q_out=q, rope=False)
    B().op_sync()
    assert got.data_ptr() == q.data_ptr() and torch.equal(q, was)            # no norm, no rotation: the same rows
    want_k, want_v = before
    want_k[table[0, 1].long(), 4:], want_v[table[0, 1].long(), 4:] = k[0, :12], v[0, :12]
    want_k[table[1, 0].long()], want_v[table[1, 0].long()] = k[1, :16], v[1, :16]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


PAGED = [  # B, T, heads, page, lens, pages per sequence
    (1, 1, 1, 16, [1], 1),
    (1, 1, 3, 64, [5000], 80),                       # one token, split and joined
    (3, 1, 2, 16, [0, 17, 300], 20),
    (2, 7, 2, 32, [129, 4000], 130),
    (1, 200, 2, 128, [777], 8),                      # a chunk: two query tiles
    (4, 130, 40, 64, [65, 1, 0, 190], 3),            # 320 units: several per stream, tails in one-tile lists
    (300, 1, 2, 16, None, 2),                        # many short sequences
    (2, 3, 1, 16, [500, 10 ** 9], 8),                # a length past the table is the table's
]


@pytest.mark.parametrize("case", PAGED)
def test_attention_paged(case):
    Bn, T, heads, page, lens, per = case
    if lens is None:
        lens = [i % (per * page + 1) for i in range(Bn)]
    kc, vc, table = cache(Bn, per, page, heads, 51)
    owned = torch.zeros(kc.shape[:2], dtype=torch.bool, device="cuda")       # what lies past the sequences is not theirs
    for b in range(Bn):
        slot = torch.arange(min(lens[b], per * page), device="cuda")
        owned[table[b].long()[slot // page], slot % page] = True
    kc[~owned], vc[~owned] = math.nan, math.inf
    q = rnd((Bn, T, heads * 128), 53)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lse = torch.full((Bn, heads, T), math.nan, device="cuda")
    out = B().op_attention_paged(q, kc, vc, table, ln, heads, lse=lse)
    B().op_sync()
    check(out, lse, *R.attention_paged(q, kc, vc, table, ln, heads))


def test_attention_paged_skips_missing_pages_and_takes_strided_caches():
    heads, page, per = 2, 16, 12
    both = rnd((40, 2, page, heads * 128), 54)          # keys and values of a page next to each other
    kc, vc = both[:, 0], both[:, 1]
    table = torch.randperm(40, generator=torch.Generator().manual_seed(55))[:per].view(1, per).to(torch.int32).cuda()
    table[0, 3], table[0, 7] = -1, 40
    q = rnd((1, 2, heads * 128), 56)
    ln = torch.tensor([per * page - 5], dtype=torch.int32, device="cuda")
    out = B().op_attention_paged(q, kc, vc, table, ln, heads)
    B().op_sync()
    check(out, None, *R.attention_paged(q, kc, vc, table, ln, heads))


def test_attention_paged_offsets_past_32_bits():
    """Pages whose elements lie past 2^31 from the cache's start."""
    heads, page = 40, 128
    pages = 2 ** 31 // (page * heads * 128) + 8
    kc = torch.zeros((pages, page, heads * 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    table = torch.tensor([[pages - 1, 0, pages - 3]], dtype=torch.int32, device="cuda")
    q, k, v = packed(1, 300, heads, 57)
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    B().op_kv_append(k, v, kc, vc, table, start, heads, (10, 10), rope=False)
    ln = torch.tensor([300], dtype=torch.int32, device="cuda")
    out = B().op_attention_paged(q[:, :2].contiguous(), kc, vc, table, ln, heads)
    B().op_sync()
    assert torch.equal(kc[pages - 1], k[0, :128]) and torch.equal(vc[pages - 3, :44], v[0, 256:])
    check(out, None, *R.attention_paged(q[:, :2], kc, vc, table, ln, heads))


def test_chunks_through_the_cache_equal_dense_attention():
    """Chunked generation: chunks of frames appended and attended one after the other; the last chunk's output is
    the dense attention over all rotated keys, the first chunk's over its own."""
    heads, hw, page, frames, chunk = 4, (6, 7), 32, 5, 2
    D, per = heads * 128, hw[0] * hw[1]
    L = frames * per
    qkv = rnd((1, L, 3 * D), 61)
    gq, gk = 1 + 0.1 * rnd((D,), 62).float(), 1 + 0.1 * rnd((D,), 63).float()
    kc, vc, table = cache(1, -(-L // page), page, heads, 64)
    kc.fill_(math.nan)
    vc.fill_(math.nan)
    outs = []
    for f0 in range(0, frames, chunk):
        n = min(chunk, frames - f0) * per
        rows = qkv[:, f0 * per:f0 * per + n]
        start = torch.tensor([f0 * per], dtype=torch.int32, device="cuda")
        q = B().op_kv_append(rows[:, :, D:2 * D], rows[:, :, 2 * D:], kc, vc, table, start, heads, hw, k_gain=gk,
                             q=rows[:, :, :D], q_gain=gq)
        outs.append(B().op_attention_paged(q, kc, vc, table, start + n, heads))
    B().op_sync()
    dense = qkv.clone().view(L, 3 * D)
    B().op_rmsnorm_rope(dense.data_ptr(), 3 * D, L, D, 1e-6, gq, rope=True, grid=(frames, *hw))
    B().op_rmsnorm_rope(dense.data_ptr() + 2 * D, 3 * D, L, D, 1e-6, gk, rope=True, grid=(frames, *hw))
    B().op_sync()
    dense = dense.view(1, L, 3 * D)
    q, k, v = dense.split(D, -1)
    one = torch.ones(1, dtype=DT, device="cuda")
    for part, rows, n in ((outs[0], slice(0, 2 * per), 2 * per), (outs[-1], slice(4 * per, L), L)):
        for h in range(heads):
            cols = slice(h * 128, (h + 1) * 128)
            ref, _, moved, size = R.attend(q[0, rows, cols].to(DT), k[0, :n, cols].to(DT), v[0, :n, cols].to(DT),
                                           one.expand(rows.stop - rows.start, n))
            # q and k of the two paths are rounded to bf16 from fp32 values that differ in their last bits: a logit
            # moves by at most 2 * 2^-8 of the sum of |q| |k| where one rounds the other way
            off = (part[0, :, cols].to(DT) - ref).abs()
            bound = 2.1 * R.HALF_STEP * (moved + ref.abs()) + 4 * R.HALF_STEP * size[:, None] * moved
            assert bool((off <= bound).all())


# ------------------------------------------------------------------ graphs, streams, repeated calls
def test_captured_and_replayed_with_new_lengths():
    heads, page, per = 2, 32, 12
    kc, vc, table = cache(2, per, page, heads, 71)
    q, k, v = packed(2, 3, heads, 72)
    qin, kin, vin = q.contiguous(), k.contiguous(), v.contiguous()
    start = torch.tensor([10, 100], dtype=torch.int32, device="cuda")
    lens = start + 3
    ws = torch.empty(max(16, B().op_attention_paged_workspace(2, heads, 3, kc, vc, table)), dtype=torch.uint8, device="cuda")
    q_out, out = torch.empty_like(qin), torch.empty_like(qin)

    def step():
        B().op_kv_append(kin, vin, kc, vc, table, start, heads, (4, 5), q=qin, q_out=q_out)
        B().op_attention_paged(q_out, kc, vc, table, lens, heads, out=out, workspace=ws)

    step()
    B().op_sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in (13, 200, 381):
        start.fill_(n)
        lens.copy_(start + 3)
        kin.copy_(rnd(kin.shape, n))
        graph.replay()
        B().op_sync()
        check(out, None, *R.attention_paged(q_out, kc, vc, table, lens, heads))
        slot = n + torch.arange(3, device="cuda")
        y, size = R.rotated(kin[1].to(DT), slot, heads, (4, 5), None)
        got = kc[table[1].long()[slot // page], slot % page].to(DT)
        assert bool(((got - y).abs() <= R.HALF_STEP * 1.001 * y.abs() + 2.0 ** -20 * size).all())


def test_two_streams_at_once_and_repeats_give_the_same_bits():
    heads, g, qb, kb = 3, (4, 9, 10), (4, 4, 8), (4, 4, 4)
    L = R.volume(g)
    sets = [packed(1, L, heads, 81 + n) for n in range(2)]
    first = []
    for q, k, v in sets:
        blocks, counts = B().op_block_select(q, k, heads, g, g, qb, kb, 4)
        first.append((blocks, counts, B().op_attention_blocks(q, k, v, heads, g, g, qb, kb, blocks, counts)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = []
        for (q, k, v), s in zip(sets, streams):
            blocks, counts = B().op_block_select(q, k, heads, g, g, qb, kb, 4, stream=s)
            got.append((blocks, counts, B().op_attention_blocks(q, k, v, heads, g, g, qb, kb, blocks, counts, stream=s)))
        torch.cuda.synchronize()
        for a, b in zip(first, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    B().op_sync()


@pytest.mark.parametrize("mode", ["blocks", "pages"])
def test_zero_wait_limit_reports_and_recovers(mode):
    heads = 12                                      # more units than streams: some waits last a unit's time
    if mode == "blocks":
        g, b = (1, 1, 1500), (1, 1, 128)
        q, k, v = packed(3, 1500, heads, 91)
        blocks, counts = lists(3, heads, 12, 12, 9, 92, False)
        run = lambda: B().op_attention_blocks(q, k, v, heads, g, g, b, b, blocks, counts)  # noqa: E731
    else:
        kc, vc, table = cache(3, 100, 32, heads, 93)
        q = rnd((3, 1100, heads * 128), 94)
        ln = torch.tensor([3111, 1700, 3200], dtype=torch.int32, device="cuda")
        run = lambda: B().op_attention_paged(q, kc, vc, table, ln, heads)  # noqa: E731
    clean = run()
    B().op_sync()
    B().op_set_wait_limit_ns(0)
    try:
        run()
        with pytest.raises(B().WanError) as e:
            B().op_sync()
        assert e.value.name == "WAN_ETIMEOUT"
    finally:
        B().op_set_wait_limit_ns(2_000_000_000)
    again = run()
    B().op_sync()
    assert torch.equal(clean, again)


@pytest.mark.parametrize("lens", [[0] * 7, [0, 0, 9000, 0, 1, 0, 0], [4000, 0, 64, 128, 1, 63, 3000], [64] * 7, [1] * 7,
                                  [100, 5000, 2000, 7000, 3, 0, 0]])
@pytest.mark.parametrize("T", [1, 140])
def test_attention_paged_ranges_cut_sequences_of_all_lengths(lens, T):
    """The tiles of all sequences are cut into even ranges: empty sequences at either end, sequences that a range
    holds whole, that several share, that end on a range's border."""
    heads, page, per = 3, 16, 563
    kc, vc, table = cache(len(lens), per, page, heads, 101)
    q = rnd((len(lens), T, heads * 128), 102)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lse = torch.full((len(lens), heads, T), math.nan, device="cuda")
    out = torch.full_like(q, math.nan)
    B().op_attention_paged(q, kc, vc, table, ln, heads, out=out, lse=lse)
    B().op_sync()
    check(out, lse, *R.attention_paged(q, kc, vc, table, ln, heads))


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e18, 1e30])
def test_block_select_at_the_ends_of_the_range(scale):
    """Products that underflow or overflow 32 bits are still ranked by their 64-bit scores."""
    heads, args = 2, ((1, 1, 256), (1, 1, 80 * 16), (1, 1, 64), (1, 1, 16))
    q, k = rnd((1, 256, 256), 111, scale), rnd((1, 1280, 256), 112, scale)
    blocks, counts = B().op_block_select(q, k, heads, *args, 9)
    B().op_sync()
    want = R.select(q, k, heads, *args, 9)
    assert torch.equal(blocks.cpu(), want[0]) and torch.equal(counts.cpu(), want[1])


def test_block_select_close_scores_are_ranked_by_their_last_bits():
    """Key blocks that differ by one bf16 step in one element of one token: far below 32-bit rounding of the
    score's sum, and more of them than one warp holds at a time."""
    nk = 300
    base = rnd((1, 16, 128), 113)
    k = base.repeat(nk, 1, 1)
    order = torch.randperm(nk, generator=torch.Generator().manual_seed(114))
    for n in range(nk):
        i = int(order[n])
        k[n, i // 128, i % 128] *= 1 + 2.0 ** -7
    k = k.reshape(1, nk * 16, 128).contiguous()
    q = rnd((1, 128, 128), 115)
    for topk in (3, 20, 150):
        args = (1, (1, 1, 128), (1, 1, nk * 16), (1, 1, 32), (1, 1, 16), topk)
        blocks, counts = B().op_block_select(q, k, *args)
        B().op_sync()
        want = R.select(q, k, *args)
        assert torch.equal(blocks.cpu(), want[0]) and torch.equal(counts.cpu(), want[1])


@pytest.mark.parametrize("nk", [2048, 2049])
def test_block_select_on_both_sides_of_the_two_stage_limit(nk):
    args = (2, (1, 1, 100), (1, 1, nk * 16), (1, 1, 32), (1, 1, 16), 77)
    q, k = rnd((1, 100, 256), 116), rnd((1, nk * 16, 256), 117)
    blocks, counts = B().op_block_select(q, k, *args)
    B().op_sync()
    want = R.select(q, k, *args)
    assert torch.equal(blocks.cpu(), want[0]) and torch.equal(counts.cpu(), want[1])


def test_kv_append_zeroes_the_rest_of_a_new_query_buffer():
    heads, page, T = 17, 32, 11
    kc, vc, table = cache(3, 2, page, heads, 121)
    q, k, v = packed(3, T, heads, 122)
    start = torch.tensor([0, 5, -2], dtype=torch.int32, device="cuda")
    count = torch.tensor([4, 0, 11], dtype=torch.int32, device="cuda")
    torch.full((3, T, heads * 128), math.nan, dtype=torch.bfloat16, device="cuda")      # memory the new buffer may take
    q_out = B().op_kv_append(k, v, kc, vc, table, start, heads, (3, 4), count=count, q=q)
    B().op_sync()
    assert bool((q_out[0, 4:] == 0).all()) and bool((q_out[1:] == 0).all())
    y, size = R.rotated(q[0, :4].to(DT), torch.arange(4, device="cuda"), heads, (3, 4), None)
    assert bool(((q_out[0, :4].to(DT) - y).abs() <= R.HALF_STEP * 1.001 * y.abs() + 2.0 ** -20 * size).all())


def test_block_select_keeps_what_large_tokens_hide():
    """Tokens of 2^30 that cancel inside a block beside ones of about 1: the scores are what the small ones leave
    (fp32 sums would lose all of them)."""
    for nk, vol in ((90, 64), (17, 16)):
        q = torch.ones((1, 64, 128), dtype=torch.bfloat16, device="cuda")
        k = torch.zeros((1, nk, vol, 128), dtype=torch.bfloat16, device="cuda")
        k[:, :, 0::4] = 2.0 ** 30
        k[:, :, 2::4] = -2.0 ** 30
        value = torch.randperm(nk, generator=torch.Generator().manual_seed(141)).to("cuda", torch.bfloat16)
        k[:, :, 1::4] = value.view(1, nk, 1, 1)
        args = (1, (1, 1, 64), (1, 1, nk * vol), (1, 1, 64), (1, 1, vol))
        blocks, counts = B().op_block_select(q, k.view(1, nk * vol, 128), *args, 5)
        B().op_sync()
        best = value.float().argsort(descending=True)[:5].sort().values.int()
        assert counts.item() == 5 and torch.equal(blocks.view(-1), best)


@pytest.mark.parametrize("nk", [30, 200])
def test_block_select_sums_past_the_range_of_fp32(nk):
    """Tokens near bf16's largest value of one sign: their sum leaves fp32's range, their mean does not."""
    q = torch.full((1, 64, 128), 2.0 ** -100, dtype=torch.bfloat16, device="cuda")
    value = (1 + torch.randperm(nk, generator=torch.Generator().manual_seed(144)) % 100 / 128).to("cuda", torch.bfloat16)
    k = torch.zeros((1, nk, 16, 128), dtype=torch.bfloat16, device="cuda")
    k[..., 0] = value.view(1, nk, 1) * 2.0 ** 127
    args = (1, (1, 1, 64), (1, 1, nk * 16), (1, 1, 64), (1, 1, 16))
    blocks, counts = B().op_block_select(q, k.view(1, nk * 16, 128), *args, 7)
    B().op_sync()
    best = value.float().argsort(descending=True, stable=True)[:7].sort().values.int()
    assert counts.item() == 7 and torch.equal(blocks.view(-1), best)

def test_join_without_parts_ends_after_the_attention():
    """Every sequence lies whole in one range, so the join kernel has nothing to do: what follows in the stream must
    still find the attention's rows."""
    heads, per, page, T = 2, 40, 64, 1
    kc, vc, table = cache(8, per, page, heads, 142)
    q = rnd((8, T, heads * 128), 143)
    ln = torch.full((8,), 64, dtype=torch.int32, device="cuda")
    assert B().op_attention_paged_workspace(8, heads, T, kc, vc, table) > 0
    out, copies = torch.empty_like(q), []
    for _ in range(20):
        out.fill_(7.0)
        B().op_attention_paged(q, kc, vc, table, ln, heads, out=out)
        copies.append(out + 0)
    B().op_sync()
    ref, ref_lse, moved, size = R.attention_paged(q, kc, vc, table, ln, heads)
    check(copies[0], None, ref, ref_lse, moved, size)
    assert all(torch.equal(c, copies[0]) for c in copies)


def test_selection_and_split_attention_captured_and_replayed():
    """Selection, then attention over few query tiles (its lists are split and joined), captured with q, k and v
    that change between replays."""
    heads, g, k3, qb, kb, topk = 2, (1, 8, 16), (6, 16, 30), (1, 8, 16), (1, 4, 8), 80
    Lk = k3[0] * k3[1] * k3[2]
    assert B().op_attention_blocks_workspace(1, heads, g, k3, qb, kb, topk) > 0
    q, k, v = rnd((1, 128, heads * 128), 151), rnd((1, Lk, heads * 128), 152), rnd((1, Lk, heads * 128), 153)

    def both():
        blocks, counts = B().op_block_select(q, k, heads, g, k3, qb, kb, topk)
        return blocks, B().op_attention_blocks(q, k, v, heads, g, k3, qb, kb, blocks, counts)

    both()
    B().op_sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for seed in (154, 155):
        for i, x in enumerate((q, k, v)):
            x.copy_(rnd(x.shape, 10 * seed + i))
        graph.replay()
        torch.cuda.synchronize()
        want = both()
        B().op_sync()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_streams_given_by_handle():
    heads, page, per, T = 2, 32, 50, 3
    kc, vc, table = cache(2, per, page, heads, 161)
    q = rnd((2, T, heads * 128), 162)
    ln = torch.tensor([1500, 40], dtype=torch.int32, device="cuda")
    want = B().op_attention_paged(q, kc, vc, table, ln, heads)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        out = B().op_attention_paged(q, kc, vc, table, ln, heads, stream=stream)
        s.synchronize()
        assert torch.equal(out, want)
    assert torch.cuda.current_stream() != s


@pytest.mark.parametrize("nk", [100, 700, 1500])
def test_block_select_with_keys_of_very_different_length(nk):
    """Blocks 10^4 times longer than the others, with scores of every size among them: the error bound of the longest
    would leave the whole row open."""
    heads, topk = 2, nk // 5
    args = (heads, (1, 1, 96), (1, 1, nk * 16), (1, 1, 32), (1, 1, 16), topk)
    q, k = rnd((1, 96, heads * 128), 171), rnd((1, nk * 16, heads * 128), 172)
    blk = k.view(nk, 16, heads * 128)
    blk[3::29] = blk[3::29] * 1e4
    blk[5::31] = blk[5::31] * 30
    blk[7] = blk[7] * 1e-6
    mask = (torch.rand((3, nk), generator=torch.Generator().manual_seed(173)) < 0.7).to(torch.uint8)
    for m in (None, mask):
        blocks, counts = B().op_block_select(q, k, *args, mask=None if m is None else m.cuda())
        B().op_sync()
        want = R.select(q, k, *args, m)
        assert torch.equal(blocks.cpu(), want[0]) and torch.equal(counts.cpu(), want[1])


@pytest.mark.parametrize("nk", [3, 13, 33, 97, 701, 1025])
@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_block_select_masks_at_any_address(nk, offset):
    """Mask rows begin at every byte of a word; bytes before and behind the mask must not count."""
    heads, topk = 1, max(1, nk // 4)
    args = (heads, (1, 1, 5 * 16), (1, 1, nk * 16), (1, 1, 16), (1, 1, 16), topk)
    q, k = rnd((1, 80, 128), 181), rnd((1, nk * 16, 128), 182)
    room = torch.full((5 * nk + 16,), 2, dtype=torch.uint8, device="cuda")
    mask = room[offset:offset + 5 * nk].view(5, nk)
    m = torch.randint(0, 8, (5, nk), generator=torch.Generator().manual_seed(183)).to(torch.uint8)
    m[m < 6] = (m[m < 6] < 3).to(torch.uint8)          # 0 and 1, some of 6 and 7: asked for
    m[4, :] = 255                                      # any value above 1 asks for a block
    mask.copy_(m)
    blocks, counts = B().op_block_select(q, k, *args, mask=mask)
    B().op_sync()
    want = R.select(q, k, *args, m.clamp(max=2))
    assert torch.equal(blocks.cpu(), want[0]) and torch.equal(counts.cpu(), want[1])


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 3])
def test_attention_paged_of_single_tokens(T, page):
    """One and two new tokens (a kernel of their own) and three: lengths around the 16 keys of a warp and the 64 of a
    tile, missing pages, foreign NaN behind the sequences, large logits, strided caches."""
    heads, per = 5, 1024 // page
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 127, 129, 500, 1023, 1024, 5000, -3]
    n = len(lens)
    room = torch.full((n * per + 2, 2, page, heads * 128 + 8), math.nan, dtype=torch.bfloat16, device="cuda")
    kc, vc = room[:, 0, :, :heads * 128], room[:, 1, :, :heads * 128]
    table = torch.randperm(n * per, generator=torch.Generator().manual_seed(191)).view(n, per).to(torch.int32).cuda()
    for b, length in enumerate(lens):
        for i in range(per):
            left = min(max(length, 0), per * page) - i * page
            if left > 0:
                p = int(table[b, i])
                kc[p, :left] = rnd((min(left, page), heads * 128), 1000 * b + i, 4.0)
                vc[p, :left] = rnd((min(left, page), heads * 128), 1000 * b + i + 500)
    table[10, ::3] = -1
    table[11, 1::2] = n * per + 2
    table[12, :] = -1                                     # nothing is there
    q = rnd((n, T, 2 * heads * 128), 192, 2.0)[..., :heads * 128]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lse = torch.empty((n, heads, T), device="cuda")
    out = B().op_attention_paged(q, kc, vc, table, ln, heads, lse=lse)
    B().op_sync()
    check(out, lse, *R.attention_paged(q, kc, vc, table, ln, heads))
    assert bool((out[12] == 0).all()) and bool(torch.isneginf(lse[12]).all())


@pytest.mark.parametrize("T", [1, 2, 3])
def test_attention_paged_infinite_logits_follow_the_formula(T):
    heads, page = 2, 32
    kc, vc, table = cache(3, 40, page, heads, 201)
    q = rnd((3, T, heads * 128), 202).abs() + 0.5
    ln = torch.tensor([1280, 1280, 1280], dtype=torch.int32, device="cuda")
    kc[int(table[0, 7]), 3, 5] = -math.inf                # head 0: weight 0
    kc[int(table[1, 9]), 30, 128 + 9] = math.inf          # head 1: inf - inf
    kc[int(table[2, 1]), 0, 3] = math.nan                 # head 0
    out = B().op_attention_paged(q, kc, vc, table, ln, heads)
    B().op_sync()
    nan = out.isnan().view(3, T, heads, 128)
    assert not bool(nan[0].any()) and bool(nan[1, :, 1].all()) and not bool(nan[1, :, 0].any())
    assert bool(nan[2, :, 0].all()) and not bool(nan[2, :, 1].any())
    kc[int(table[0, 7]), 3, 5] = -3e4                     # as far down as it matters
    kc[int(table[1, 9]), 30, 128 + 9] = 0
    kc[int(table[2, 1]), 0, 3] = 0
    ref = R.attention_paged(q, kc, vc, table, ln, heads)
    check(out[:1], None, *(x[:1] for x in ref))


@pytest.mark.parametrize("T", [1, 2])
def test_attention_paged_of_many_sequences(T):
    """More lists than units that fill the GPU, of all lengths from none to three pages."""
    n, heads, page = 270, 3, 32
    kc, vc, table = cache(n, 3, page, heads, 211)
    q = rnd((n, T, heads * 128), 212)
    ln = (torch.arange(n, dtype=torch.int32) * 7 % 97).cuda()
    lse = torch.empty((n, heads, T), device="cuda")
    out = B().op_attention_paged(q, kc, vc, table, ln, heads, lse=lse)
    B().op_sync()
    check(out, lse, *R.attention_paged(q, kc, vc, table, ln, heads))
