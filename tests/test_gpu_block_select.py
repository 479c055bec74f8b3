"""Block selection on the GPU at the sizes of its kernels for large grids: means of many blocks (one group of
threads per column slice) and rows of more than 2048 key blocks (64-bit scores throughout)."""
import math

import pytest
import torch

from tests import attention_parts as R
from tests.gpu_common import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    from video_diffusion_transformer_dit_b200 import binding
    binding.lib()


def rnd(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def check(q, k, heads, qg, kg, qb, kb, topk, mask=None):
    from video_diffusion_transformer_dit_b200 import binding
    args = (q, k, heads, qg, kg, qb, kb, topk)
    blocks, counts = binding.op_block_select(*args, mask=None if mask is None else mask.cuda())
    binding.op_sync()
    want = R.select_rows(*args, mask)
    assert torch.equal(counts.cpu(), want[1])
    assert torch.equal(blocks.cpu(), want[0])
    return blocks, counts


# ------------------------------------------------------------------ means of many blocks
def many(B, heads, qg, kg, qb, kb):
    """From about 9500 blocks times heads times samples on, an SM has its threads without four groups per slice."""
    return (R.block_count(qg, qb) + R.block_count(kg, kb)) * heads * 16 * B >= 148 * 1024


MANY = [  # B, heads, q grid, k grid, q block, k block, topk
    (1, 12, (1, 1, 3190), (1, 1, 16 * 800 - 5), (1, 1, 64), (1, 1, 16), 90),
    (2, 17, (6, 29, 31), (8, 29, 31), (3, 5, 7), (2, 2, 4), 33),      # 105-token blocks, a column slice that is not full
    (1, 40, (8, 33, 37), (8, 33, 37), (4, 4, 8), (4, 4, 4), 23),
    (1, 13, (3, 50, 61), (3, 50, 61), (1, 8, 16), (1, 8, 2), 400),    # cut to 2, 3 and 1 columns or rows
    (1, 5, (1, 1, 700), (1, 1, 2048 * 16), (1, 1, 10), (1, 1, 16), 300),
    (3, 9, (1, 1, 500), (1, 1, 128 * 380 - 127), (1, 1, 77), (1, 1, 128), 50),   # the last block holds one token
    (1, 1, (1, 1, 9400), (1, 1, 1500), (1, 1, 1), (1, 1, 16), 11),    # one query per block, one head
]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("case", MANY)
def test_means_of_many_blocks(case, masked):
    B, heads, qg, kg, qb, kb, topk = case
    assert many(B, heads, qg, kg, qb, kb)
    mask = None
    if masked:
        g = torch.Generator().manual_seed(3)
        mask = torch.randint(0, 5, (R.block_count(qg, qb), R.block_count(kg, kb)), generator=g).clamp(max=1).to(torch.uint8)
        mask[:, 5::97] = 2
    qkv = rnd((B, max(R.volume(qg), R.volume(kg)), 2 * heads * 128), 1)         # column slices of wider rows
    if qg == kg:
        q, k = qkv.split(heads * 128, -1)
    else:
        q, k = rnd((B, R.volume(qg), heads * 128), 2), rnd((B, R.volume(kg), heads * 128), 3)
    check(q, k, heads, qg, kg, qb, kb, topk, mask)


@pytest.mark.parametrize("vol", [16, 64, 128])
def test_means_of_many_blocks_keep_what_large_tokens_hide(vol):
    """Tokens of 2^30 that cancel inside a block beside ones of about 1, at every place of the block."""
    heads, nk = 12, 900
    assert many(1, heads, (1, 1, 64), (1, 1, nk * vol), (1, 1, 64), (1, 1, vol))
    q = torch.ones((1, 64, heads * 128), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((1, nk, vol, heads * 128), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(141)
    rank = torch.rand((heads, nk), generator=g).argsort(-1)
    value = (rank % 256).to("cuda", torch.bfloat16).repeat_interleave(128, 0).T                 # exact in bf16
    for j in range(nk):
        large, other, small = torch.randperm(vol, generator=g)[:3].tolist()
        k[0, j, large], k[0, j, other] = 2.0 ** 30, -2.0 ** 30
        k[0, j, small] = value[j]
    blocks, _ = check(q, k.view(1, nk * vol, heads * 128), heads, (1, 1, 64), (1, 1, nk * vol), (1, 1, 64), (1, 1, vol), 5)
    for h in range(heads):
        best = (-(rank[h] % 256)).argsort(stable=True)[:5].sort().values.int()
        assert torch.equal(blocks[0, h, 0].cpu(), best)


def test_means_of_many_blocks_whose_sums_leave_fp32():
    heads, nk = 12, 900
    q = torch.full((1, 64, heads * 128), 2.0 ** -100, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((1, nk, 16, heads, 128), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(144)
    value = (1 + torch.rand((nk, heads), generator=g).argsort(0) % 100 / 128).to("cuda", torch.bfloat16)
    k[0, ..., 0] = value.view(nk, 1, heads) * 2.0 ** 127
    blocks, _ = check(q, k.view(1, nk * 16, heads * 128), heads, (1, 1, 64), (1, 1, nk * 16), (1, 1, 64), (1, 1, 16), 7)
    for h in range(heads):
        best = value[:, h].float().argsort(descending=True, stable=True)[:7].sort().values.int()
        assert torch.equal(blocks[0, h, 0], best)


# ------------------------------------------------------------------ rows of more than 2048 key blocks
LONG = [2049, 2300, 5000, 12288 + 77]


@pytest.mark.parametrize("nk", LONG)
@pytest.mark.parametrize("topk", [1, 255, 1000, 2049])
def test_long_rows(nk, topk):
    q, k = rnd((2, 75, 3 * 128), 11), rnd((2, nk * 16 - 9, 3 * 128), 12)
    check(q, k, 3, (1, 1, 75), (1, 1, nk * 16 - 9), (1, 1, 2), (1, 1, 16), topk)


def test_the_longest_row():
    nk = 28800
    q, k = rnd((1, 96, 128), 13), rnd((1, nk * 16, 128), 14)
    mask = torch.ones((3, nk), dtype=torch.uint8)
    mask[1, ::3] = 0
    mask[2, 100:28700] = 0
    mask[2, 28799] = 2
    for topk in (1, 500, 9600):
        check(q, k, 1, (1, 1, 96), (1, 1, nk * 16), (1, 1, 32), (1, 1, 16), topk, mask)
    blocks, _ = check(q, k, 1, (1, 1, 96), (1, 1, nk * 16), (1, 1, 32), (1, 1, 16), nk)
    assert torch.equal(blocks[0, 0, 1].cpu(), torch.arange(nk, dtype=torch.int32))


@pytest.mark.parametrize("nk", LONG)
@pytest.mark.parametrize("topk", [7, 300])
def test_long_rows_with_masks_that_leave_them_empty_short_and_full(nk, topk):
    heads = 2
    q, k = rnd((1, 9 * 32, heads * 128), 15), rnd((1, nk * 16, heads * 128), 16)
    mask = torch.ones(9, nk, dtype=torch.uint8)
    mask[0] = 0                                  # nothing
    mask[1] = 0
    mask[1, [nk - 1, 3, 257]] = 1                # fewer than topk
    mask[2, :1000] = 2                           # more asked for than topk: the lowest blocks
    mask[3, nk - 3:] = 255                       # some asked for, the rest by score
    mask[4, ::2] = 0
    mask[5] = 2                                  # all
    mask[6] = 0
    mask[6, 250:250 + topk] = 2                  # exactly topk, over the border of 256
    mask[7] = 0
    mask[7, nk - topk:] = 1
    mask[8] = torch.randint(0, 6, (nk,), generator=torch.Generator().manual_seed(17)).to(torch.uint8)
    mask[8][mask[8] > 2] = 1
    _, counts = check(q, k, heads, (1, 1, 288), (1, 1, nk * 16), (1, 1, 32), (1, 1, 16), topk, mask)
    assert counts[0, 0].tolist() == [0, 3] + [topk] * 7


@pytest.mark.parametrize("nk", LONG)
@pytest.mark.parametrize("topk", [3, 257, 1025])
def test_long_rows_give_equal_scores_to_the_lowest_blocks(nk, topk):
    """Five key blocks over and over, with whole numbers (their scores are exact): a border among equals that lie
    in every piece of 256; and a row of zeros alone."""
    g = torch.Generator(device="cuda").manual_seed(18)
    pattern = torch.randint(-8, 9, (5, 16, 128), generator=g, device="cuda").bfloat16()
    k = pattern[torch.randint(0, 5, (nk,), generator=g, device="cuda")].reshape(1, nk * 16, 128).contiguous()
    q = torch.randint(-8, 9, (1, 48, 128), generator=g, device="cuda").bfloat16()
    q[0, 32:] = 0
    blocks, _ = check(q, k, 1, (1, 1, 48), (1, 1, nk * 16), (1, 1, 16), (1, 1, 16), topk)
    assert blocks[0, 0, 2].tolist() == list(range(topk))


@pytest.mark.parametrize("nk", LONG)
def test_long_rows_rank_nan_and_infinite_scores(nk):
    q, k = rnd((1, 16, 128), 19).abs(), rnd((1, nk * 16, 128), 20)
    for at, value in ((5, math.nan), (9, math.inf), (11, -math.inf), (300, math.inf), (nk - 1, math.nan), (600, -math.inf)):
        k[0, at * 16 + 2, 7] = value
    mask = torch.ones((1, nk), dtype=torch.uint8)
    mask[0, [9, 600]] = 0
    for topk in (1, 2, nk - 5, nk - 1, nk):
        blocks, _ = check(q, k, 1, (1, 1, 16), (1, 1, nk * 16), (1, 1, 16), (1, 1, 16), topk)
        assert 9 in blocks[0, 0, 0].tolist() and (topk == 1 or 300 in blocks[0, 0, 0].tolist())
        check(q, k, 1, (1, 1, 16), (1, 1, nk * 16), (1, 1, 16), (1, 1, 16), topk, mask)
    q[0, 3, 0] = math.nan                        # every score of the row
    blocks, counts = check(q, k, 1, (1, 1, 16), (1, 1, nk * 16), (1, 1, 16), (1, 1, 16), 400)
    assert int(counts) == 400 and blocks[0, 0, 0].tolist() == list(range(400))


@pytest.mark.parametrize("scale", [1e-30, 1e18, 1e30])
def test_long_rows_at_the_ends_of_the_range(scale):
    q, k = rnd((1, 64, 128), 21, scale), rnd((1, 2100 * 16, 128), 22, scale)
    check(q, k, 1, (1, 1, 64), (1, 1, 2100 * 16), (1, 1, 16), (1, 1, 16), 99)


# ------------------------------------------------------------------ rows of every length that a kernel is built for
@pytest.mark.parametrize("nk", [n + d for n in (128, 256, 384, 512, 640, 768, 896, 1024, 1536, 2048) for d in (-31, 0, 1)])
def test_rows_around_each_kernels_length(nk):
    heads, topk = 2, nk // 6
    args = (heads, (1, 1, 6 * 16), (1, 1, nk * 16), (1, 1, 16), (1, 1, 16))
    q, k = rnd((1, 96, heads * 128), 31), rnd((1, nk * 16, heads * 128), 32)
    k[0, 16:16 * (nk // 2), :128] = k[0, :16, :128].repeat(nk // 2 - 1, 1)      # head 0: half of the blocks are equal
    k[0, 16 * (nk - 3):16 * (nk - 2)] *= 100
    check(q, k, *args, topk)
    mask = torch.randint(0, 5, (6, nk), generator=torch.Generator().manual_seed(33)).clamp(max=1).to(torch.uint8)
    mask[1] = 0
    mask[1, nk - 1] = 1
    mask[2, -topk - 3:] = 2
    mask[3, ::7] = 2
    check(q, k, *args, topk, mask)
    check(q, k, *args, nk, mask)
    k[0, 16 * (nk - 1) + 3, 130] = math.nan                                     # head 1
    check(q, k, *args, topk, mask)
