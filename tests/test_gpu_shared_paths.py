"""xmla_decode_shared on both sides of its dispatch borders: every test says which
kernels it means to reach and checks, by the workspace the call asks for, that it
does."""
import pytest
import torch

from mla_latent_kv_yarn_b200 import seq_parallel as sp
from mla_latent_kv_yarn_b200 import session, xmla
import shared_cases as sc
from gpu_cases import cfgs

pytestmark = pytest.mark.gpu

PAGE, ROW_BYTES = sc.PAGE, 2 * sc.ROW


def copies_prefix(batch, q_len, pages, longest):
    """Whether the call shares the prefix (its workspace then grows by the fp16 copy of
    every further prefix page: 302 MB for 4,096 of them) instead of attending each
    sequence whole (partials of at most one split per SM: under 10 MB)."""
    f, n = xmla.xmla_decode_shared_workspace_size, session.num_sms()
    more = f(batch, q_len, pages + 4096, longest + 4096 * PAGE, n) - f(batch, q_len, pages, longest, n)
    return more >= 4096 * PAGE * ROW_BYTES


def run(st, prefix, q, longest, cfg, dec=None):
    dec = dec or session.SharedDecoder(q.shape[0], q.shape[1], prefix.numel(), longest, q.device)
    out = dec.decode(cfg, st, prefix, q, xmla.xmla_softmax_scale(xmla.xmla_yarn_default(), 192))
    torch.cuda.synchronize()
    return out, dec


# ---------------------------------------------------------------- NaN and infinity

@pytest.mark.parametrize("value,column", [("nan", 17), ("nan", 511), ("nan", 570), ("inf", 300), ("-inf", 0)])
@pytest.mark.parametrize("batch,q_len,pages,room,shares", [
    (4, 1, 30, 0, False), (1, 1, 30, 0, False), (2, 2, 1, 0, False), (1, 3, 700, 0, False),
    (6, 1, 30, 0, True), (3, 2, 30, 50000, True)])
def test_a_row_that_is_no_number_reaches_the_output(batch, q_len, pages, room, shares, value, column):
    cfg, ocfg = cfgs()
    own = [70 + 9 * b for b in range(batch)]
    st, prefix, q, longest = sc.shared_state(batch, q_len, pages, own, seed=60, room=room)
    assert copies_prefix(batch, q_len, pages, longest) == shares
    ref = sc.shared_reference(st, prefix, q, ocfg)
    block = st.block_table[batch - 1, pages].long()  # a token of the last sequence's own
    kept = st.pool[block, 9].clone()
    st.pool[block, 9, column] = float(value)
    out, dec = run(st, prefix, q, longest, cfg)
    assert dec.check_status() == 0
    assert torch.isnan(out[-1]).all()
    if batch > 1:
        sc.assert_decode_close(out[:-1], ref[:-1])
    st.pool[block, 9] = kept
    st.pool[prefix[pages // 2].long(), 3, column] = float(value)  # a token of everyone's
    out, dec = run(st, prefix, q, longest, cfg)
    assert dec.check_status() == 0
    assert torch.isnan(out).all()


@pytest.mark.parametrize("q_len,seqlens", [(1, [5000, 300]), (1, [200, 100, 70, 90] * 50), (4, [5000, 300]),
                                           (16, [3000, 300]), (100, [700, 300])])
def test_a_nan_row_reaches_the_output_of_the_plain_decode(q_len, seqlens):
    """The same rule in xmla_decode: splits merged by the combine, and prompt chunks."""
    cfg, ocfg = cfgs()
    own = [n - PAGE for n in seqlens]
    st, prefix, q, longest = sc.shared_state(len(own), q_len, 1, own, seed=61)
    st.block_table[:, :1] = torch.arange(len(own), device="cuda", dtype=torch.int32)[:, None] + st.num_blocks
    st.pool = torch.cat([st.pool, st.pool[:1].expand(len(own), -1, -1)])
    st.num_blocks += len(own)
    dec = session.Decoder(len(own), q_len, longest, "cuda")
    scale = xmla.xmla_softmax_scale(cfg, 192)
    whole = dec.decode(cfg, st, q, scale).clone()
    st.pool[st.block_table[1, 0].long(), 9, 17] = float("nan")
    out = dec.decode(cfg, st, q, scale)
    torch.cuda.synchronize()
    assert dec.check_status() == 0 and torch.isfinite(whole).all()
    assert torch.isnan(out[1]).all()
    others = [b for b in range(len(own)) if b != 1]
    assert torch.equal(out[others], whole[others])


def test_a_nan_row_reaches_the_output_of_a_sharded_decode():
    cfg, ocfg = cfgs()
    st, prefix, q, longest = sc.shared_state(2, 1, 1, [3000, 900], seed=62)
    st.block_table[:, :1] = prefix
    st.pool[st.block_table[0, 40].long(), 9, 17] = float("nan")  # on the last rank
    world, partials = 3, []
    for rank in range(world):
        d = sp.ShardDecoder(2, 1, longest, world, rank, "cuda")
        d.decode_shard(cfg, sp.shard_layer(st, d.page_lo, d.page_hi), q, xmla.xmla_softmax_scale(cfg, 192))
        torch.cuda.synchronize()
        assert int(d.status.item()) == 0
        partials.append(d.partial)
    d.gathered.copy_(torch.cat(partials))
    out = d.combine(st.W_UV)
    torch.cuda.synchronize()
    assert torch.isnan(out[0]).all()
    sc.assert_decode_close(out[1:], sc.shared_reference(st, prefix, q, ocfg)[1:])
