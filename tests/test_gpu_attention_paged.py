"""Attention over a paged cache on the GPU, for each of its kernels (one and two new tokens, and more): every value
row with its own weight, bounds without the rounding of p where p stays in 32 bits, offsets past 32 bits, many
sequences, joins without parts, NaN."""
import math

import pytest
import torch

from tests import attention_parts as R
from tests.gpu_common import DT, need_gpu
from tests.test_gpu_attention_parts import cache, check, lists, packed, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    from video_diffusion_transformer_dit_b200 import binding
    binding.lib()


def B():
    from video_diffusion_transformer_dit_b200 import binding
    return binding


def per_head(x, heads):
    return x.unflatten(-1, (heads, 128)).transpose(1, 2)


def check_single(out, lse, ref, ref_lse, moved, size, keys):
    h = ref_lse.shape[1]
    R.check_rows(per_head(out, h), lse, per_head(ref, h), ref_lse, per_head(moved, h), per_head(size, h)[..., 0], keys)
    assert bool((out[(ref_lse == -math.inf).transpose(1, 2).repeat_interleave(128, -1)] == 0).all())


# ------------------------------------------------------------------ every key with its own weight
MARKED = [  # page, lens
    (16, [1900]), (64, [1900]), (128, [1, 64, 65, 1500, 0, 129]), (32, [700] * 5), (16, [33] * 40)]


@pytest.mark.parametrize("T", [1, 2, 3, 140])
@pytest.mark.parametrize("page,lens", MARKED)
def test_every_cached_value_counts_once_with_its_keys_weight(page, lens, T):
    heads, n = 3, len(lens)
    per = -(-max(lens) // page) + 1
    kc, vc, table = cache(n, per, page, heads, 301)
    kc.fill_(math.nan)
    vc.fill_(math.nan)
    g = torch.Generator(device="cuda").manual_seed(302)
    b = torch.randint(0, 7, (n, per * page), generator=g, device="cuda")
    there = torch.arange(per * page, device="cuda") < torch.tensor(lens, device="cuda")[:, None]
    weight = torch.where(there, 2.0 ** -b.to(DT), 0.0)
    slot = torch.arange(per * page, device="cuda").expand(n, -1)[there]
    at = table.long().repeat_interleave(page, 1)[there], slot % page
    kc[at] = R.marked_keys(b, heads)[there]
    q = R.marked_query((n, T, heads * 128), "cuda")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for first in range(0, max(lens), 128):
        vc[at] = R.marked_values(per * page, first, heads, "cuda").expand(n, -1, -1)[there]
        out = B().op_attention_paged(q, kc, vc, table, ln, heads)
        B().op_sync()
        R.check_marked(out.view(n, T, heads, 128), weight[:, None, None], first)


@pytest.mark.parametrize("case", [
    (2, (3, 8, 8), (7, 9, 20), (1, 8, 8), (2, 4, 4), 40),         # whole lists
    (1, (1, 1, 50), (1, 1, 1900), (1, 1, 64), (1, 1, 64), 30),    # split lists
    (1, (2, 9, 9), (5, 9, 13), (3, 5, 7), (1, 8, 16), 9),         # 128 keys to a block
    (1, (1, 8, 16), (9, 10, 11), (1, 8, 16), (1, 4, 4), 70)])     # 16, split
def test_every_listed_value_counts_with_its_keys_weight(case):
    Bn, qg, kg, qb, kb, topk = case
    heads, nk, Lk, Lq = 2, R.block_count(kg, kb), R.volume(kg), R.volume(qg)
    blocks, counts = lists(Bn, heads, R.block_count(qg, qb), nk, topk, 303)
    blocks[0, 0, 0, 1] = blocks[0, 0, 0, 0]                       # listed twice
    g = torch.Generator(device="cuda").manual_seed(304)
    b = torch.randint(0, 7, (Lk,), generator=g, device="cuda")
    k = R.marked_keys(b, heads).expand(Bn, -1, -1).contiguous()
    q = R.marked_query((Bn, Lq, heads * 128), "cuda")
    there = torch.arange(topk, device="cuda") < counts[..., None]
    times = torch.zeros((Bn, heads, blocks.shape[2], nk + 1), dtype=DT, device="cuda")
    times.scatter_add_(-1, torch.where(there, blocks, nk).long(), torch.ones_like(there, dtype=DT))
    weight = times[:, :, R.block_of(qg, qb, "cuda")][..., R.block_of(kg, kb, "cuda")] * 2.0 ** -b.to(DT)
    for first in range(0, Lk, 128):
        v = R.marked_values(Lk, first, heads, "cuda").expand(Bn, -1, -1).contiguous()
        out = B().op_attention_blocks(q, k, v, heads, qg, kg, qb, kb, blocks, counts)
        B().op_sync()
        R.check_marked(out.view(Bn, Lq, heads, 128), weight.transpose(1, 2), first)


# ------------------------------------------------------------------ p in 32 bits
@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("page,lens,heads", [(64, [5000], 3), (16, [0, 17, 300, 4097], 2), (128, [9000, 1, 2, 8000], 1),
                                             (32, [130] * 270, 2), (16, [i % 33 for i in range(300)], 2)])
def test_one_and_two_tokens_keep_their_probabilities_in_32_bits(page, lens, heads, T):
    per = -(-max(lens) // page)
    kc, vc, table = cache(len(lens), per, page, heads, 311)
    q = rnd((len(lens), T, heads * 128), 312, 2.0)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lse = torch.empty((len(lens), heads, T), device="cuda")
    out = B().op_attention_paged(q, kc, vc, table, ln, heads, lse=lse)
    B().op_sync()
    check_single(out, lse, *R.attention_paged(q, kc, vc, table, ln, heads), max(lens))


# ------------------------------------------------------------------ both kernels over the same range
@pytest.mark.parametrize("T", [1, 2, 3, 140])
def test_pages_past_32_bits(T):
    """Pages whose elements lie past 2^31 from the cache's start."""
    heads, page = 40, 128
    pages = 2 ** 31 // (page * heads * 128) + 8
    kc = torch.zeros((pages, page, heads * 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    table = torch.tensor([[pages - 1, 0, pages - 3]], dtype=torch.int32, device="cuda")
    q, k, v = packed(1, 300, heads, 321)
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    B().op_kv_append(k, v, kc, vc, table, start, heads, (10, 10), rope=False)
    ln = torch.tensor([300], dtype=torch.int32, device="cuda")
    q = q[:, :T].contiguous()
    out = B().op_attention_paged(q, kc, vc, table, ln, heads)
    B().op_sync()
    check(out, None, *R.attention_paged(q, kc, vc, table, ln, heads))


@pytest.mark.parametrize("T", [1, 2, 3, 130])
@pytest.mark.parametrize("n", [257, 300, 600])
def test_more_sequences_than_one_launch_takes(n, T):
    """Launches of 256 sequences after each other, the last one's few lists split, in one workspace."""
    heads, page, per = 2, 32, 12
    kc, vc, table = cache(n, per, page, heads, 331)
    table = torch.cat((table, torch.full_like(table, -7)), 1)[:, :per]          # rows further apart than they are long
    q = rnd((n, T, 3 * heads * 128), 332)[..., heads * 128:2 * heads * 128]
    ln = (torch.arange(n, dtype=torch.int32) * 89 % (per * page + 1)).cuda()
    ln[100:110] = 0
    ln[-1] = per * page
    assert B().op_attention_paged_workspace(n, heads, T, kc, vc, table) > 0
    lse = torch.full((n, heads, T), math.nan, device="cuda")
    room = torch.full((n * T + 2, heads * 128 + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    out = room[:n * T].view(n, T, -1)[..., :heads * 128]
    B().op_attention_paged(q, kc, vc, table, ln, heads, out=out, lse=lse)
    B().op_sync()
    ref = R.attention_paged(q, kc, vc, table, ln, heads)
    if T <= 2:
        check_single(out, lse, *ref, per * page)
    else:
        check(out, lse, *ref)
    assert bool((room[n * T:] == 7).all()) and bool((room[:, heads * 128:] == 7).all())


@pytest.mark.parametrize("T", [2, 3, 140])
def test_joins_without_parts_end_after_the_attention(T):
    """Every sequence lies whole in one range, so the join kernel has nothing to do: what follows in the stream must
    still find the attention's rows."""
    heads, per, page = 2, 40, 64
    kc, vc, table = cache(8, per, page, heads, 341)
    q = rnd((8, T, heads * 128), 342)
    ln = torch.full((8,), 64, dtype=torch.int32, device="cuda")
    assert B().op_attention_paged_workspace(8, heads, T, kc, vc, table) > 0
    out, copies = torch.empty_like(q), []
    for _ in range(20):
        out.fill_(7.0)
        B().op_attention_paged(q, kc, vc, table, ln, heads, out=out)
        copies.append(out + 0)
    B().op_sync()
    check(copies[0], None, *R.attention_paged(q, kc, vc, table, ln, heads))
    assert all(torch.equal(c, copies[0]) for c in copies)


@pytest.mark.parametrize("T", [1, 2, 3])
def test_nan_of_a_query_or_of_all_keys_of_a_page_reaches_the_row(T):
    heads, page, per = 2, 16, 20
    kc, vc, table = cache(2, per, page, heads, 351)
    q = rnd((2, T, heads * 128), 352)
    ln = torch.tensor([300, 16], dtype=torch.int32, device="cuda")
    q[0, T - 1, 5] = math.nan
    lse = torch.empty((2, heads, T), device="cuda")
    out = B().op_attention_paged(q, kc, vc, table, ln, heads, lse=lse)
    B().op_sync()
    want = torch.zeros((2, heads, T), dtype=torch.bool, device="cuda")
    want[0, 0, T - 1] = True
    assert torch.equal(lse.isnan(), want) and torch.equal(out.isnan(), want.transpose(1, 2).repeat_interleave(128, -1))
    q[0, T - 1, 5] = 0
    kc[table[0, 1].long(), :, 128 + 7] = math.nan         # 16 keys that one warp has alone
    kc[table[1, 0].long(), :, 7] = math.nan               # all there are
    out = B().op_attention_paged(q, kc, vc, table, ln, heads, lse=lse)
    B().op_sync()
    want[:] = False
    want[0, 1], want[1, 0] = True, True
    assert torch.equal(lse.isnan(), want) and torch.equal(out.isnan(), want.transpose(1, 2).repeat_interleave(128, -1))
