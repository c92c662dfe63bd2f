"""xmla_decode_shared on both sides of its dispatch borders: every test says which
kernels it means to reach and checks, by the workspace the call asks for, that it
does."""
import pytest
import torch

from mla_latent_kv_yarn_b200 import seq_parallel as sp
from mla_latent_kv_yarn_b200 import session, xmla
from oracle import mla_oracle as om
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


def copies_own(batch, q_len, pages, longest):
    """Whether the own parts (of more than 256 + q_len tokens of room) are copied too."""
    f, n = xmla.xmla_decode_shared_workspace_size, session.num_sms()
    return f(batch, q_len, pages, longest, n) - f(batch, q_len, pages, longest - 256, n) >= batch * 256 * ROW_BYTES


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


# ---------------------------------------------------------------- scores that rise late

# Every 256 tokens hold one token of each size in turn: a row's maximum rises by far
# more than its lazy border of 8 (log2 units) in the second and third block of three,
# wherever a run's segment begins.
SIZES = (2.0, 8.0, 30.0)


def rising_state(batch, q_len, pages, own, seed):
    st, prefix, q, longest = sc.shared_state(batch, q_len, pages, own, seed=seed, scale=0.3)
    for k in range(pages * PAGE // 256):
        t = 256 * k + (37 * k + 11) % 256
        st.pool[prefix[t // PAGE].long(), t % PAGE] *= SIZES[k % 3]
    for b, n in enumerate(own):
        for k in range((n - q_len + 1) // 256):
            t = 256 * k + (53 * k + 29) % 256
            st.pool[st.block_table[b, pages + t // PAGE].long(), t % PAGE] *= SIZES[k % 3]
    return st, prefix, q, longest


def bound_and_reference(st, prefix, q, ocfg, few):
    """(|out - reference| at most, reference, whether each row's maximum rises late).

    As in shared_cases.shared_error_bound, with what these states add:
    E: scores off by 2^-11 (fp16 query; with few queries hi + lo parts, 2^-16) and
       2^-14 (float32 sums) of their sum of magnitudes change the output by at most
       (e^(2E) - 1) sum p |v - o|.
    Probabilities rounded to fp16: 2^-11 sum p |v| and, below 2^-14, half a step of
       2^-24: 2^-25 against a sum of at least 2^7 (the reference maximum's own), 2^-32
       max |v| per token.  Rounded to bf16 (few queries: all tokens, summed as rounded):
       2^-8 sum p |v - o|.
    Accumulation in float32 over a segment of at most 10 blocks, 160 steps of 2^-23
       each: under 2^-15 sum p |v|.
    Merged rows as two bf16 parts: 2^-16 sum_c |x_c W_UV[c]|; output rounded to bf16:
       2^-8 of the value and of the errors before it."""
    B, J = q.shape[:2]
    n0 = prefix.numel() * PAGE
    scale = om.softmax_scale(ocfg)
    wk, wv = st.W_UK.double(), st.W_UV.double()
    ref = torch.zeros(B, J, sc.H, sc.V, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(ref)
    late = torch.zeros(B, J, sc.H, dtype=torch.bool, device=q.device)
    head = st.pool[prefix.long()].reshape(n0, sc.ROW).double()
    for b in range(B):
        n = int(st.seqlens[b])
        rows = torch.cat([head, st.pool[sc.own_table(st, b, prefix, n)].reshape(-1, sc.ROW)[:n - n0].double()])
        pos = torch.arange(n - J, n, device=q.device)
        hidden = torch.arange(n, device=q.device)[None] > pos[:, None]
        for h in range(sc.H):
            x = q[b, :, h].double()
            x = torch.cat([x[:, :sc.NOPE] @ wk[h], sc.rotated(x[:, sc.NOPE:], pos, ocfg)], -1) * scale
            s = (x @ rows.T).masked_fill(hidden, -torch.inf)
            top = s[:, :n0 // 256 * 256].reshape(J, -1, 256).amax(-1) / torch.log(torch.tensor(2.0))
            late[b, :, h] = (top[:, 1:] > top[:, :-1] + 10).any(-1)
            p = torch.softmax(s, -1)
            v = rows[:, :sc.LATENT] @ wv[h]
            o = p @ v
            ref[b, :, h] = o
            E = ((2.0 ** -16 if few else 2.0 ** -11) + 2.0 ** -14) * (x.abs() @ rows.abs().T).amax(-1)
            parts = 2.0 ** -16 * ((p @ rows[:, :sc.LATENT]).abs() @ wv[h].abs())
            pv = p @ v.abs()
            for j in range(J):
                away = (p[j, :, None] * (v - o[j]).abs()).sum(0)
                e = torch.expm1(2 * E[j]) * away + 2.0 ** -15 * pv[j] + parts[j]
                if few:
                    e = e + 2.0 ** -8 * away
                else:
                    e = e + 2.0 ** -11 * pv[j] + n * 2.0 ** -32 * v.abs().amax(0)
                bound[b, j, h] = e + 2.0 ** -8 * (o[j].abs() + e) + 1e-6
    return bound, ref, late


@pytest.mark.parametrize("batch,q_len,pages,own,shares", [
    (4, 1, 192, [3, 300, 64, 700], False),
    (6, 1, 640, [3, 1200, 64, 700, 1, 1279], True),
    (3, 2, 640, [2, 1200, 700], True),
    (40, 1, 256, [1 + 19 * b for b in range(40)], True),
    (5, 8, 192, [8, 1200, 700, 300, 999], True)])
def test_scores_that_rise_late(batch, q_len, pages, own, shares):
    cfg, ocfg = cfgs()
    st, prefix, q, longest = rising_state(batch, q_len, pages, own, seed=30 + batch)
    assert copies_prefix(batch, q_len, pages, longest) == shares
    if shares:
        assert copies_own(batch, q_len, pages, longest)
        # every run holds four blocks and more: one of each size behind its first
        tiles = -(-batch * q_len * sc.H // 128)
        assert tiles * (pages // 4 + 1) >= 4 * (session.num_sms() // 2)
    out, dec = run(st, prefix, q, longest, cfg)
    assert dec.check_status() == 0
    bound, ref, late = bound_and_reference(st, prefix, q, ocfg, few=not shares)
    assert float(late.double().mean()) > 0.9
    over = float(((out.double() - ref).abs() - bound).max())
    assert over <= 0.0, over
    # the bound says something: a result without the rescale would be off by the
    # size of the output
    assert float(bound.norm() / ref.norm()) < 0.5


# ---------------------------------------------------------------- bad block ids

SHARES = [(3, 1, False), (6, 1, True), (3, 4, True), (40, 1, True)]


@pytest.mark.parametrize("batch,q_len,shares", SHARES)
def test_bad_prefix_block(batch, q_len, shares):
    cfg, ocfg = cfgs()
    st, prefix, q, longest = sc.shared_state(batch, q_len, 6, [q_len + (13 * b) % 90 for b in range(batch)], seed=40)
    assert copies_prefix(batch, q_len, 6, longest) == shares
    zeroed = session.LayerState(**{**st.__dict__, "pool": st.pool.clone()})
    zeroed.pool[prefix[4].long()] = 0
    ref = sc.shared_reference(zeroed, prefix, q, ocfg)
    for bad in (-1, st.num_blocks, 2 ** 31 - 1, -2 ** 31):
        broken = prefix.clone()
        broken[4] = bad
        out, dec = run(st, broken, q, longest, cfg)
        assert dec.check_status() == 5
        sc.assert_decode_close(out, ref, f"block {bad}")


@pytest.mark.parametrize("room", [400, 100000])
@pytest.mark.parametrize("batch,q_len,shares", SHARES)
def test_bad_own_block(batch, q_len, shares, room):
    cfg, ocfg = cfgs()
    own = [q_len + (13 * b) % 90 for b in range(batch)]
    own[1] = 350
    st, prefix, q, longest = sc.shared_state(batch, q_len, 6, own, seed=41, room=room)
    assert copies_prefix(batch, q_len, 6, longest) == shares
    assert copies_own(batch, q_len, 6, longest) == (shares and room == 400)
    zeroed = session.LayerState(**{**st.__dict__, "pool": st.pool.clone()})
    zeroed.pool[st.block_table[1, 8].long()] = 0
    ref = sc.shared_reference(zeroed, prefix, q, ocfg)
    for bad in (-1, st.num_blocks, 2 ** 31 - 1, -2 ** 31):
        table = st.block_table.clone()
        table[1, 8] = bad
        out, dec = run(session.LayerState(**{**st.__dict__, "block_table": table}), prefix, q, longest, cfg)
        assert dec.check_status() == 5
        sc.assert_decode_close(out, ref, f"block {bad}")


# ---------------------------------------------------------------- one buffer, several plans

def test_one_workspace_for_calls_of_different_sizes():
    """A large batch, a smaller one, few queries and the large one again in the same
    buffer: each finds the tables and partials of the call before it."""
    cfg, ocfg = cfgs()
    sizes = [(130, 1, 5, [1 + 2 * b for b in range(130)], 0), (6, 2, 9, [2, 70, 300, 64, 5, 2], 0),
             (2, 1, 9, [2, 500], 0), (6, 1, 3, [1, 2, 3, 4, 5, 6], 60000),
             (1, 1, 1, [1], 0), (130, 1, 5, [261 - 2 * b for b in range(130)], 0)]
    states = [sc.shared_state(b, j, pages, own, seed=50 + i, room=room)
              for i, (b, j, pages, own, room) in enumerate(sizes)]
    decs = [session.SharedDecoder(q.shape[0], q.shape[1], prefix.numel(), longest, "cuda")
            for st, prefix, q, longest in states]
    buffer = torch.full((max(d.ws_bytes for d in decs),), 0xFF, dtype=torch.uint8, device="cuda")
    for d in decs:
        d.workspace = buffer
    scale = xmla.xmla_softmax_scale(cfg, 192)
    for d, (st, prefix, q, longest) in zip(decs, states):  # one right behind the other
        d.decode(cfg, st, prefix, q, scale)
    torch.cuda.synchronize()
    for i, (d, (st, prefix, q, longest)) in enumerate(zip(decs, states)):
        assert d.check_status() == 0
        sc.assert_decode_close(d.out, sc.shared_reference(st, prefix, q, ocfg), f"call {i}")


@pytest.mark.parametrize("batch", [5, 6, 7, 8, 9, 11, 13, 15, 16, 17, 31, 33, 47, 48, 49, 127, 128, 129, 137])
def test_every_remainder_of_output_rows(batch):
    """Numbers of queries that leave the W_UV kernel's warps at different rows, and its
    boxes of eight rows partly filled; nothing behind the last row is written."""
    cfg, ocfg = cfgs()
    st, prefix, q, longest = sc.shared_state(batch, 1, 2, [1 + (5 * b) % 70 for b in range(batch)], seed=70 + batch)
    dec = session.SharedDecoder(batch, 1, 2, longest, "cuda")
    out = torch.full((batch + 2, 1, 32, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    dec.decode(cfg, st, prefix, q, xmla.xmla_softmax_scale(cfg, 192), out=out)
    torch.cuda.synchronize()
    assert dec.check_status() == 0 and bool((out[batch:] == 7.0).all())
    sc.assert_decode_close(out[:batch], sc.shared_reference(st, prefix, q, ocfg))
