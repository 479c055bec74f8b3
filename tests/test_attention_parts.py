"""Refusals and sizes of the attention operators over parts of the sequence: every check runs before the device
is looked for, so they are tested without one."""
import ctypes as C

import pytest

EINVAL, ESHAPE = 1, 2
FAKE = C.c_void_p(1 << 20)          # never dereferenced: every call below is refused first
ODD = C.c_void_p((1 << 20) + 8)     # not 16-byte aligned
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from video_diffusion_transformer_dit_b200 import binding, build
    build.build()
    return binding.lib()


def grid(q=(3, 8, 8), k=(3, 8, 8), qb=(1, 8, 8), kb=(1, 4, 4)):
    from video_diffusion_transformer_dit_b200 import binding
    return binding._block_grid(q, k, qb, kb)


def cache(k=FAKE, v=FAKE, page_stride=64 * 256, token_stride=256, num_pages=10, page_size=64, table=FAKE, table_ld=4,
          max_pages=4):
    from video_diffusion_transformer_dit_b200 import binding
    return binding.wan_kv_cache(k, v, page_stride, token_stride, num_pages, page_size, table, table_ld, max_pages)


BAD_GRIDS = [dict(q=(0, 8, 8)), dict(k=(3, -1, 8)), dict(qb=(1, 0, 8)), dict(kb=(0, 4, 4)),
             dict(qb=(3, 8, 8)),                  # 192 queries per block
             dict(kb=(1, 3, 5)), dict(kb=(1, 2, 4)), dict(kb=(4, 8, 8)),   # 15, 8, 256 keys
             dict(q=(1 << 12, 1 << 12, 1 << 12))]


def test_block_select_refuses(lib):
    ok = dict(q=FAKE, ldq=256, k=FAKE, ldk=256, B=1, heads=2, g=grid(), mask=None, topk=3, blocks=FAKE, counts=FAKE,
              ws=FAKE, nbytes=BIG)

    def call(**kw):
        a = {**ok, **kw}
        g = a["g"]
        return lib.wan_op_block_select(a["q"], a["ldq"], a["k"], a["ldk"], a["B"], a["heads"], C.byref(g) if g else None,
                                       a["mask"], a["topk"], a["blocks"], a["counts"], a["ws"], a["nbytes"], None)

    for name in ("q", "k", "g", "blocks", "counts", "ws"):
        assert call(**{name: None}) == EINVAL, name
    for g in BAD_GRIDS:
        assert call(g=grid(**g)) == ESHAPE, g
        assert lib.wan_op_block_select_workspace(1, 2, C.byref(grid(**g))) == -1
    for kw in (dict(B=-1), dict(heads=0), dict(B=300, heads=300), dict(ldq=255), dict(ldq=248), dict(ldk=260), dict(topk=0),
               dict(topk=13), dict(q=ODD), dict(k=ODD), dict(ws=ODD), dict(nbytes=100),
               dict(g=grid(q=(1, 1, 64), k=(1, 1, 16 * 28801), qb=(1, 1, 64), kb=(1, 1, 16)))):
        assert call(**kw) == ESHAPE, kw
    assert call(B=0) == 0
    need = lib.wan_op_block_select_workspace(1, 2, C.byref(grid()))
    assert need > 0 and call(nbytes=need - 1) == ESHAPE
    assert lib.wan_op_block_select_workspace(1, 2, None) == -1


def test_attention_blocks_refuses(lib):
    ok = dict(q=FAKE, ldq=256, k=FAKE, ldk=256, v=FAKE, ldv=256, o=FAKE, ldo=256, B=1, heads=2, g=grid(), blocks=FAKE,
              counts=FAKE, topk=3, lse=None, ws=FAKE, nbytes=BIG)

    def call(**kw):
        a = {**ok, **kw}
        g = a["g"]
        return lib.wan_op_attention_blocks(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["o"], a["ldo"], a["B"],
                                           a["heads"], C.byref(g) if g else None, a["blocks"], a["counts"], a["topk"],
                                           a["lse"], a["ws"], a["nbytes"], None)

    for name in ("q", "k", "v", "o", "g", "blocks", "counts"):
        assert call(**{name: None}) == EINVAL, name
    for g in BAD_GRIDS:
        assert call(g=grid(**g)) == ESHAPE, g
        assert lib.wan_op_attention_blocks_workspace(1, 2, C.byref(grid(**g)), 3) == -1
    for kw in (dict(B=-1), dict(heads=-2), dict(ldq=128), dict(ldk=257), dict(ldv=0), dict(ldo=252), dict(topk=0), dict(q=ODD),
               dict(k=ODD), dict(v=ODD), dict(o=ODD)):
        assert call(**kw) == ESHAPE, kw
    assert call(B=0) == 0
    # few query tiles and a long list: the list is split, and the parts need room
    long = grid(q=(1, 1, 1), k=(1, 1, 64000), qb=(1, 1, 128), kb=(1, 1, 64))
    need = lib.wan_op_attention_blocks_workspace(1, 2, C.byref(long), 1000)
    assert need > 0
    assert call(g=long, topk=1000, ws=None) == EINVAL and call(g=long, topk=1000, nbytes=need - 1) == ESHAPE
    assert call(g=long, topk=1000, ws=ODD) == ESHAPE
    assert lib.wan_op_attention_blocks_workspace(1, 2, C.byref(long), 0) == -1


BAD_CACHES = [dict(page_size=0), dict(page_size=48), dict(page_size=256), dict(num_pages=0), dict(max_pages=0),
              dict(max_pages=5), dict(token_stride=248), dict(token_stride=252), dict(page_stride=63 * 256),
              dict(page_stride=64 * 256 + 4), dict(k=ODD), dict(v=ODD), dict(max_pages=1 << 25, table_ld=1 << 25)]


def test_kv_append_refuses(lib):
    ok = dict(k=FAKE, ldk=256, v=FAKE, ldv=256, B=2, T=3, heads=2, start=FAKE, count=None, k_gain=None, rope=1, H=4, W=5,
              split=(44, 42, 42), theta=1e4, q=FAKE, ldq=256, q_gain=None, q_out=FAKE, ldqo=256, c=cache())

    def call(**kw):
        a = {**ok, **kw}
        c = a["c"]
        return lib.wan_op_kv_append(a["k"], a["ldk"], a["v"], a["ldv"], a["B"], a["T"], a["heads"], a["start"], a["count"],
                                    a["k_gain"], 1e-6, a["rope"], a["H"], a["W"], *a["split"], a["theta"], a["q"], a["ldq"],
                                    a["q_gain"], a["q_out"], a["ldqo"], 0, C.byref(c) if c else None, None)

    for kw in (dict(k=None), dict(v=None), dict(start=None), dict(c=None), dict(q_out=None), dict(c=cache(k=None)),
               dict(c=cache(v=None)), dict(c=cache(table=None))):
        assert call(**kw) == EINVAL, kw
    for c in BAD_CACHES:
        assert call(c=cache(**c)) == ESHAPE, c
    for kw in (dict(B=-1), dict(T=-1), dict(heads=0), dict(heads=3), dict(heads=97, ldk=12416, ldv=12416, ldq=12416, ldqo=12416, c=cache(token_stride=12416, page_stride=64 * 12416)), dict(ldk=128), dict(ldv=252), dict(ldq=0), dict(ldqo=260),
               dict(k=ODD), dict(v=ODD), dict(q=ODD), dict(q_out=ODD), dict(k_gain=ODD), dict(q_gain=ODD), dict(H=0), dict(W=-1),
               dict(split=(44, 42, 41)), dict(split=(43, 43, 42)), dict(split=(130, -2, 0)), dict(theta=0.0),
               dict(theta=float("nan"))):
        assert call(**kw) == ESHAPE, kw
    assert call(B=0) == 0 and call(T=0) == 0


def test_attention_paged_refuses(lib):
    ok = dict(q=FAKE, ldq=256, c=cache(), lens=FAKE, o=FAKE, ldo=256, B=2, heads=2, T=3, lse=None, ws=FAKE, nbytes=BIG)

    def call(**kw):
        a = {**ok, **kw}
        c = a["c"]
        return lib.wan_op_attention_paged(a["q"], a["ldq"], C.byref(c) if c else None, a["lens"], a["o"], a["ldo"], a["B"],
                                          a["heads"], a["T"], a["lse"], a["ws"], a["nbytes"], None)

    for kw in (dict(q=None), dict(o=None), dict(lens=None), dict(c=None), dict(c=cache(k=None)), dict(c=cache(table=None))):
        assert call(**kw) == EINVAL, kw
    for c in BAD_CACHES:
        assert call(c=cache(**c)) == ESHAPE, c
        assert lib.wan_op_attention_paged_workspace(2, 2, 3, C.byref(cache(**c))) == -1
    for kw in (dict(B=-1), dict(T=-1), dict(heads=0), dict(heads=3), dict(ldq=128), dict(ldo=252), dict(q=ODD), dict(o=ODD)):
        assert call(**kw) == ESHAPE, kw
    assert call(B=0) == 0 and call(T=0) == 0
    c = cache(max_pages=1000, table_ld=1000)
    need = lib.wan_op_attention_paged_workspace(1, 2, 1, C.byref(c))
    assert need > 0
    assert call(B=1, T=1, c=c, ws=None) == EINVAL and call(B=1, T=1, c=c, nbytes=need - 1) == ESHAPE


def test_python_wrappers_refuse_tensors_that_do_not_fit():
    import torch
    from video_diffusion_transformer_dit_b200 import binding
    x = torch.zeros(1, 192, 256, dtype=torch.bfloat16)      # not on a GPU
    with pytest.raises(ValueError):
        binding.op_block_select(x, x, 2, (3, 8, 8), (3, 8, 8), (1, 8, 8), (1, 4, 4), 3)
    i = torch.zeros(1, 2, 3, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.op_attention_blocks(x, x, x, 2, (3, 8, 8), (3, 8, 8), (1, 8, 8), (1, 4, 4), i, i[..., 0])
    c = torch.zeros(4, 16, 256, dtype=torch.bfloat16)
    t = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.op_attention_paged(x, c, c, t, t[0, :1], 2)
    with pytest.raises(ValueError):
        binding.op_kv_append(x, x, c, c, t, t[0, :1], 2, (8, 8))


def test_lists_beyond_the_index_range_are_refused(lib):
    g = grid()
    for topk in ((1 << 24) + 1, 1 << 30, (1 << 31) - 1):
        assert lib.wan_op_attention_blocks_workspace(1, 2, C.byref(g), topk) == -1
        assert lib.wan_op_attention_blocks(FAKE, 256, FAKE, 256, FAKE, 256, FAKE, 256, 1, 2, C.byref(g), FAKE, FAKE, topk,
                                           None, FAKE, BIG, None) == ESHAPE
    assert lib.wan_op_attention_blocks_workspace(1, 2, C.byref(g), 1 << 24) >= 0


def test_python_wrappers_refuse_grids_and_streams_that_do_not_fit(lib):
    import types

    import torch
    from video_diffusion_transformer_dit_b200 import binding
    for d in (((8, 8), (3, 8, 8), (1, 8, 8), (1, 4, 4)), ((3, 8, 8, 1), (3, 8, 8), (1, 8), (1, 4, 4)),
              ((3, 8, 8), (3, 8, 8), (1, 8, 8), (16,))):
        with pytest.raises(ValueError, match="frames, rows, columns"):
            binding.op_block_select_workspace(1, 2, *d)
    with pytest.raises(ValueError, match="stream of cuda:0"):
        binding._torch()
        binding._elsewhere(torch.device("cuda", 0), types.SimpleNamespace(device=torch.device("cuda", 1)))


def test_append_refuses_more_rows_than_its_grid_holds(lib):
    c = cache()
    for B, T in ((1, (1 << 29) + 1), (1 << 15, 1 << 15)):
        assert lib.wan_op_kv_append(FAKE, 256, FAKE, 256, B, T, 2, FAKE, None, None, 1e-6, 0, 0, 0, 0, 0, 0, 1e4, None, 0, None,
                                    None, 0, 0, C.byref(c), None) == ESHAPE


@pytest.mark.parametrize("B,heads", [(1, 1), (1, 32), (2, 40)])
@pytest.mark.parametrize("g", [dict(q=(1, 1, 64), k=(1, 1, 16 * 28801), qb=(1, 1, 64), kb=(1, 1, 16)),      # key blocks
                               dict(q=(1, 1, 65535 * 32 + 1), k=(1, 1, 64), qb=(1, 1, 1), kb=(1, 1, 16)),   # query blocks
                               # with 32 heads the bytes of its scores are 2^64 and more
                               dict(q=(1, 1, 1 << 30), k=(1, 1, 1 << 30), qb=(1, 1, 1), kb=(1, 1, 16))])
def test_block_select_names_no_workspace_for_grids_it_refuses(lib, g, B, heads):
    g = grid(**g)
    assert lib.wan_op_block_select_workspace(B, heads, C.byref(g)) == -1
    assert lib.wan_op_block_select(FAKE, 128 * heads, FAKE, 128 * heads, B, heads, C.byref(g), None, 1, FAKE, FAKE, FAKE, BIG,
                                   None) == ESHAPE


def test_block_select_names_a_workspace_for_the_largest_grid_it_takes(lib):
    g = grid(q=(1, 1, 65535 * 32), k=(1, 1, 16 * 28800), qb=(1, 1, 1), kb=(1, 1, 16))
    assert lib.wan_op_block_select_workspace(1, 512, C.byref(g)) > 65535 * 32 * 28800 * 512 * 8


def test_python_selection_refuses_sizes_by_their_own_status(lib, monkeypatch):
    """A box, a grid or a topk outside the limits is WAN_ESHAPE, not the null workspace that the wrapper has for it,
    and nothing is allocated for it."""
    import torch
    from video_diffusion_transformer_dit_b200 import binding
    monkeypatch.setattr(binding, "_elsewhere", lambda device, stream: None)      # host tensors: refused all the same
    x = torch.zeros(1, 192, 12 * 128, dtype=torch.bfloat16)
    room = torch.zeros(1 << 20, dtype=torch.uint8)
    for kb, topk in (((1, 3, 5), 3), ((1, 4, 4), 0), ((1, 4, 4), -1), ((1, 4, 4), 13), ((1, 4, 4), (1 << 31) - 1),
                     ((1, 4, 4), (1 << 32) + 3)):
        for workspace in (None, room):
            with pytest.raises(binding.WanError) as e:
                binding.op_block_select(x, x, 12, (3, 8, 8), (3, 8, 8), (1, 8, 8), kb, topk, workspace=workspace)
            assert e.value.name == "WAN_ESHAPE", (kb, topk)


@pytest.mark.parametrize("masked", [False, True])
def test_the_two_selections_of_the_oracle_agree(masked):
    import math

    import torch
    from tests import attention_parts as R
    g = torch.Generator().manual_seed(7)
    for qg, kg, qb, kb, topk in (((3, 8, 8), (3, 8, 8), (1, 8, 8), (1, 4, 4), 5), ((2, 5, 9), (7, 9, 20), (4, 4, 8), (2, 4, 4), 11),
                                 ((1, 1, 40), (1, 1, 16 * 90 - 3), (1, 1, 32), (1, 1, 16), 30)):
        q = torch.randn((2, R.volume(qg), 256), generator=g).bfloat16()
        k = torch.randn((2, R.volume(kg), 256), generator=g).bfloat16()
        k[1, 16:48] = 0                                     # equal scores
        k[1, 100, 3], k[1, 120, 130] = math.nan, math.inf
        mask = torch.randint(0, 4, (R.block_count(qg, qb), R.block_count(kg, kb)), generator=g).to(torch.uint8) if masked else None
        a = R.select(q, k, 2, qg, kg, qb, kb, topk, mask)
        b = R.select_rows(q, k, 2, qg, kg, qb, kb, topk, mask)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
