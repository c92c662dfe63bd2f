"""Norms of vectors whose squares leave the range of float32: values beside the largest
and the smallest bf16 ones, with and without an eps, against 64 bits.

A bf16 result is one rounding (2^-8 of the value, and half of bf16's smallest step,
2^-134) of float32 arithmetic, which adds under 2^-18 of the vector's largest value
(as in test_gpu_norm.py; scaling by a power of two is exact)."""
import numpy as np
import pytest
import torch

from mla_latent_kv_yarn_b200 import session, xmla
import shared_cases as sc
from gpu_cases import cfgs

pytestmark = pytest.mark.gpu

HALF, SLACK, TINY = 2.0 ** -8, 2.0 ** -18, 2.0 ** -134
# a vector of each of these times N(0, 1), one head each
SCALES = [1.0, 1e20, 3e-25, 1.0, 2e37, 1e-39, 7e17, 1e-19, 4e-23, 5e18, 1.0, 0.0]


def vectors(g, rows, dim):
    """[rows, len(SCALES) + 2, dim]: and one large value among ordinary ones, one
    ordinary among small ones."""
    x = torch.randn(rows, len(SCALES) + 2, dim, generator=g, device="cuda", dtype=torch.float64)
    x[:, :-2] *= torch.tensor(SCALES, dtype=torch.float64, device="cuda")[:, None]
    x[:, -2, dim // 3] = 1e30
    x[:, -1] *= 1e-30
    x[:, -1, dim // 2] = 1e-21
    return x.to(torch.bfloat16)


def assert_rounded(got, ref, what):
    """ref rounded once, NaN where ref is."""
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    ref, got = torch.nan_to_num(ref), torch.nan_to_num(got).double()
    top = ref.abs().amax(-1, keepdim=True)
    over = (got - ref).abs() - HALF * ref.abs() - SLACK * top - TINY
    assert float(over.max()) <= 0.0, f"{what}: {float(over.max()):.3e}"


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-34, 1e-42, 3e38])
@pytest.mark.parametrize("dim,offset", [(192, 128), (64, 0), (256, 192), (66, 1), (200, 136), (512, 448), (1023, 700),
                                        (1024, 960)])
def test_norm_rope_over_the_whole_range(dim, offset, eps):
    cfg, ocfg = cfgs()
    g = torch.Generator(device="cuda")
    g.manual_seed(dim)
    x, w = vectors(g, 5, dim), sc.randn(g, dim)
    R, H, D = x.shape
    pos = torch.randint(0, 2 ** 20, (R,), generator=g, device="cuda")
    eps64 = float(np.float32(eps))
    plain = sc.normed(x, w, eps64)
    turned = plain.clone()
    turned[..., offset:offset + 64] = sc.rotated(plain[..., offset:offset + 64], pos[:, None], ocfg)
    for rotate, ref in ((True, turned), (False, plain)):
        out, own = torch.full_like(x, 7.0), x.clone()
        for dst, src in ((out, x), (own, own)):  # and in place
            xmla.xmla_norm_rope(cfg if rotate else None, src, H * D, D, dst, H * D, D, R, H, D, w, 0, eps, offset,
                                pos)
        torch.cuda.synchronize()
        for h in range(H):
            assert_rounded(out[:, h], ref[:, h], f"head {h}, rotate {rotate}")
        assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(own))
    # a head does not depend on its neighbours: the ordinary ones are those of a call by
    # themselves, bit for bit
    usual = [0, 3, 10]
    alone = torch.empty(R, 3, D, dtype=torch.bfloat16, device="cuda")
    xmla.xmla_norm_rope(None, x[:, usual].contiguous(), 3 * D, D, alone, 3 * D, D, R, 3, D, w, 0, eps)
    torch.cuda.synchronize()
    assert torch.equal(out[:, usual], alone)


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("with_pe", [True, False])
@pytest.mark.parametrize("cache", ["bf16", "q8"])
def test_normed_append_over_the_whole_range(cache, with_pe, eps):
    cfg, ocfg = cfgs()
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    lat = vectors(g, 1, 512)[0, :-3]  # (without the zero vector, whose norm with no eps is NaN,
    pe = vectors(g, 1, 64)[0, :-3]    # and the mixed ones, which leave the 8-bit format's range)
    lat, pe = lat[:-1], pe[:-1]
    n = lat.shape[0]
    T = 2 * n + 1
    lat = torch.cat([lat, lat.flip(0), lat[:1]])
    pe = torch.cat([pe, pe, pe[:1]]) if with_pe else sc.randn(g, T, 64)
    kv = torch.cat([lat, pe], 1).contiguous()
    w_kv, w_pe = (1 + 0.1 * torch.randn(k, generator=g, device="cuda") for k in (512, 64))
    w_kv, w_pe = w_kv.bfloat16(), w_pe.bfloat16() if with_pe else None
    st = session.LayerState(pool=session.new_pool_q8(2, "cuda") if cache == "q8" else session.new_pool(2, "cuda"),
                            block_table=torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), seqlens=None,
                            W_UK=None, W_UV=None, num_blocks=2, max_blocks=2, cache=cache)
    pos = torch.arange(T, device="cuda") + 50
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    session.append_normed_rows(cfg, st, kv, w_kv, w_pe, eps, pos, ids, status)
    eps64 = float(np.float32(eps))
    ref = torch.cat([sc.normed(lat, w_kv, eps64),
                     sc.rotated(sc.normed(pe, w_pe, eps64) if with_pe else pe.double(), pos, ocfg)], -1)
    if cache == "bf16":
        got = st.pool[st.block_table[0, pos // 64].long(), pos % 64]
        assert_rounded(got[:, :512], ref[:, :512], "latent")
        assert_rounded(got[:, 512:], ref[:, 512:], "rope key")
    else:
        got = torch.empty(T, 576, dtype=torch.bfloat16, device="cuda")
        xmla.xmla_cache_read_q8(st.pool, 2, st.block_table, 2, 1, ids, pos, T, got, 576, status)
        # a code is a rounding to half a unit of its block; float32's slack may move the
        # block's largest value across a power of two or a value across a tie
        unit = torch.exp2(torch.ceil(torch.log2(ref.reshape(T, 18, 32).abs().amax(-1, keepdim=True)
                                                * (1 + SLACK) / 127)).clamp(-14, 8)).expand(T, 18, 32).reshape(T, 576)
        top = torch.cat([ref[:, :512].abs().amax(-1, keepdim=True).expand(-1, 512),
                         ref[:, 512:].abs().amax(-1, keepdim=True).expand(-1, 64)], -1)
        assert float(((got.double() - ref).abs() - unit / 2 - SLACK * top).max()) <= 0.0
    torch.cuda.synchronize()
    assert int(status) == 0


def test_codes_are_the_nearest_up_to_float32():
    """|x / unit - code| is at most a half, up to the error of x: the squares' sum takes
    32 + 4 steps of 2^-24, of which the factor has half, its own rounding and the
    refinement's rest one each, the product one more: under 21 x 2^-24 < 2^-19."""
    cfg, _ = cfgs()
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    T = 4096
    kv, w = sc.randn(g, T, 576, std=3.0), (1 + 0.1 * torch.randn(512, generator=g, device="cuda")).bfloat16()
    blocks = T // 64
    st = session.LayerState(pool=session.new_pool_q8(blocks, "cuda"),
                            block_table=torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)[None],
                            seqlens=None, W_UK=None, W_UV=None, num_blocks=blocks, max_blocks=blocks, cache="q8")
    pos, ids = torch.arange(T, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    session.append_normed_rows(cfg, st, kv, w, None, 1e-6, pos, ids)
    rows = st.pool[st.block_table[0].long()].reshape(T, 608)
    codes = rows[:, :512].view(torch.int8).double().reshape(T, 16, 32)
    unit = torch.exp2(rows[:, 576:592].view(torch.int8).double())[..., None]
    x = sc.normed(kv[:, :512], w, float(np.float32(1e-6))).reshape(T, 16, 32) / unit
    assert float(((x - codes).abs() - 0.5 - x.abs() * 2.0 ** -19).max()) <= 0.0
    # and the unit is the smallest that holds the block
    top = x.abs().amax(-1)
    assert float(top.max()) <= 127 * (1 + 2.0 ** -19) and float(top.min()) >= 63.5 * (1 - 2.0 ** -19)


@pytest.mark.parametrize("cache", ["bf16", "q8"])
def test_large_weights_meet_large_values(cache):
    """x w alone would leave float32's range; the result does not."""
    g = torch.Generator(device="cuda")
    g.manual_seed(10)
    T = 20
    scale = torch.tensor([1e16, 1e-14, 1.0, 3e17, 1e-10] * 4, device="cuda")[:, None]
    kv = (torch.randn(T, 576, generator=g, device="cuda") * scale).bfloat16()
    w = torch.randn(512, generator=g, device="cuda").double() * (1e25 if cache == "bf16" else 1e-2)
    w[::3] *= 1e-30 if cache == "bf16" else 1.0
    w = w.bfloat16()
    st = session.LayerState(pool=session.new_pool_q8(1, "cuda") if cache == "q8" else session.new_pool(1, "cuda"),
                            block_table=torch.zeros(1, 1, dtype=torch.int32, device="cuda"), seqlens=None, W_UK=None,
                            W_UV=None, num_blocks=1, max_blocks=1, cache=cache)
    pos, ids = torch.arange(T, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    session.append_normed_rows(None, st, kv, w, None, 0.0, pos, ids)
    ref = sc.normed(kv[:, :512], w, 0.0)
    if cache == "bf16":
        got = st.pool[0, :T, :512]
        assert torch.isfinite(got).all()
        over = (got.double() - ref).abs() - (HALF + SLACK) * ref.abs() - TINY
    else:
        got = torch.empty(T, 576, dtype=torch.bfloat16, device="cuda")
        xmla.xmla_cache_read_q8(st.pool, 1, st.block_table, 1, 1, ids, pos, T, got, 576)
        unit = torch.exp2(st.pool[0, :T, 576:592].view(torch.int8).double())[..., None].expand(T, 16, 32).reshape(T, 512)
        over = (got[:, :512].double() - ref).abs() - unit / 2 - SLACK * ref.abs()
    assert float(over.max()) <= 0.0
