"""The model's forward with its self-attention over selected key blocks: the staged calls of one rank hand out each
block's normed and rotated q, k, v, and take back the attention's output."""
import pytest
import torch

from oracle import wan_oracle as O
from tests import attention_parts as R
from tests.gpu_common import make_dit, need_gpu, rel_l2

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def staged(dit, lat, t, ctx, attend):
    """wan_dit_forward by its stages, with attend(block, q, k, v) for the self-attention."""
    from video_diffusion_transformer_dit_b200 import ulysses as U
    rank = U.SpRank(dit, 0, 1)
    rank.begin(lat, t, ctx)
    for i in range(dit.cfg["num_blocks"]):
        q, k, v = rank.block_qkv(i).view(rank.B, rank.L, 3 * rank.hd).split(rank.hd, -1)
        rank.block_finish(i, attend(i, q, k, v))
    vel = rank.end()
    dit.sync()
    return vel


@pytest.mark.parametrize("per_token", [False, True])
def test_forward_with_attention_over_selected_blocks(per_token):
    from video_diffusion_transformer_dit_b200 import binding, configs, synth
    cfg = configs.model_config("wan2.1-1.3b", num_blocks=2)
    shape, grid, qb, kb, heads = (2, 16, 3, 14, 18), (3, 7, 9), (1, 4, 8), (1, 4, 4), 12
    L, nk = R.volume(grid), R.block_count(grid, kb)
    W = {n: w.cuda() for n, w in synth.make_weights(cfg, seed=51).items()}
    lat = synth.make_latent(shape, seed=51).cuda()
    ctx = synth.make_context(2, 24, cfg["text_dim"], seed=51).cuda()
    t = synth.make_timestep_per_token(2, L, 7 * 9, seed=51).cuda() if per_token else torch.tensor([999.0, 500.0]).cuda()
    assert O.token_count(*shape[2:]) == L
    dit = make_dit(cfg, 2, L, 24, W)

    def sparse(topk, kept):
        def attend(i, q, k, v):
            kept.append(binding.op_block_select(q, k, heads, grid, grid, qb, kb, topk))
            return binding.op_attention_blocks(q, k, v, heads, grid, grid, qb, kb, *kept[-1])
        return attend

    # all blocks kept: the forward itself, up to the attention's own roundings
    dense = dit.forward(lat, t, ctx, sync=True)
    vel = staged(dit, lat, t, ctx, sparse(nk, []))
    assert rel_l2(vel, dense) < 1e-2
    # a third of them: the same stages with the attention over the same lists in 64 bits
    kept = []
    vel = staged(dit, lat, t, ctx, sparse(nk // 3, kept))
    assert all(bool((c == nk // 3).all()) for _, c in kept)
    exact = staged(dit, lat, t, ctx, lambda i, q, k, v: R.attention_blocks(
        q, k, v, heads, grid, grid, qb, kb, *kept[i])[0].to(torch.bfloat16))
    assert rel_l2(vel, exact) < 1e-2 < rel_l2(vel, dense)
    again = staged(dit, lat, t, ctx, sparse(nk // 3, []))
    assert torch.equal(again, vel)
