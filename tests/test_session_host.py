"""What the session helpers refuse before any library call: nothing here needs a GPU
(tensors live on the CPU, and a call that got as far as the library would fail there)."""
import pytest
import torch

from mla_latent_kv_yarn_b200 import build as xbuild

xbuild.build()

from mla_latent_kv_yarn_b200 import session, xmla  # noqa: E402


@pytest.fixture(autouse=True)
def no_library_call(monkeypatch):
    """Any library call ends the test: it must have been refused before."""
    def called():
        raise AssertionError("reached the library")
    monkeypatch.setattr(xmla, "lib", called)


def state(cache="bf16", blocks=8, batch=2, pages=4):
    pool = session.new_pool_q8(blocks, "cpu") if cache == "q8" else session.new_pool(blocks, "cpu")
    table = torch.arange(batch * pages, dtype=torch.int32).view(batch, pages) % blocks
    return session.LayerState(pool=pool, block_table=table,
                              seqlens=torch.full((batch,), 70, dtype=torch.int32),
                              W_UK=torch.zeros(32, 128, 512, dtype=torch.bfloat16),
                              W_UV=torch.zeros(32, 512, 128, dtype=torch.bfloat16), num_blocks=blocks,
                              max_blocks=pages, cache=cache)


def shared_decoder(batch=2, q_len=1, prefix_pages=1, max_seqlen=256):
    d = object.__new__(session.SharedDecoder)  # (the constructor asks the device for its size)
    d.batch, d.q_len, d.prefix_pages, d.max_seqlen = batch, q_len, prefix_pages, max_seqlen
    d.ws_bytes = 1024
    d.workspace = torch.zeros(1024, dtype=torch.uint8)
    d.out = torch.zeros(batch, q_len, 32, 128, dtype=torch.bfloat16)
    d.status = torch.zeros(1, dtype=torch.int32)
    return d


def test_shared_decode_refuses_an_8bit_cache():
    q = torch.zeros(2, 1, 32, 192, dtype=torch.bfloat16)
    prefix = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="bf16 cache"):
        shared_decoder().decode(None, state("q8"), prefix, q, 0.1)
    with pytest.raises(AssertionError, match="reached the library"):
        shared_decoder().decode(None, state("bf16"), prefix, q, 0.1)


def test_read_back_refuses_a_bf16_cache():
    with pytest.raises(ValueError, match="8-bit cache"):
        session.read_back_q8(state("bf16"), [70, 70])


def refused(f, match):
    with pytest.raises(ValueError, match=match):
        f()


def reaches(f):
    with pytest.raises(AssertionError, match="reached the library"):
        f()


@pytest.mark.parametrize("cache", ["bf16", "q8"])
def test_append_normed_rows_refuses_what_it_would_misread(cache):
    st, T, bf = state(cache), 3, torch.bfloat16
    good = dict(kv=torch.zeros(T, 576, dtype=bf), kv_weight=torch.ones(512, dtype=bf),
                pe_weight=torch.ones(64, dtype=bf), positions=torch.zeros(T, dtype=torch.int64),
                seq_ids=torch.zeros(T, dtype=torch.int32))

    def call(**over):
        a = {**good, **over}
        session.append_normed_rows(None, st, a["kv"], a["kv_weight"], a["pe_weight"], 1e-6, a["positions"],
                                   a["seq_ids"])

    reaches(call)
    reaches(lambda: call(pe_weight=None))
    reaches(lambda: call(kv=torch.zeros(T, 640, dtype=bf)[:, :576]))
    reaches(lambda: call(kv=torch.zeros(T, 640, dtype=bf)[:, 64:]))
    reaches(lambda: call(positions=torch.zeros(T + 1, dtype=torch.int64)))
    refused(lambda: call(kv=torch.zeros(T, 1152, dtype=bf)[..., ::2]), "adjacent")
    refused(lambda: call(kv=torch.zeros(576, T, dtype=bf).t()), "adjacent")
    refused(lambda: call(kv=torch.zeros(T, 512, dtype=bf)), "576")
    refused(lambda: call(kv=torch.zeros(T, 576)), "kv must")
    refused(lambda: call(kv_weight=torch.ones(1024, dtype=bf)[::2]), "kv_weight")
    refused(lambda: call(kv_weight=torch.ones(511, dtype=bf)), "kv_weight")
    refused(lambda: call(kv_weight=torch.ones(512)), "kv_weight")
    refused(lambda: call(pe_weight=torch.ones(128, dtype=bf)[::2]), "pe_weight")
    refused(lambda: call(pe_weight=torch.ones(32, dtype=bf)), "pe_weight")
    refused(lambda: call(positions=torch.zeros(T, dtype=torch.int32)), "positions")
    refused(lambda: call(positions=torch.zeros(T - 1, dtype=torch.int64)), "positions")
    refused(lambda: call(positions=torch.zeros(2 * T, dtype=torch.int64)[::2]), "positions")
    refused(lambda: call(seq_ids=torch.zeros(T, dtype=torch.int64)), "seq_ids")
    refused(lambda: call(seq_ids=torch.zeros(T - 1, dtype=torch.int32)), "seq_ids")


def test_a_single_row_of_any_stride_is_appended(monkeypatch):
    """torch gives a dimension of one any stride; the library wants a row's pitch."""
    seen = {}
    monkeypatch.setattr(xmla, "xmla_cache_append_norm",
                        lambda *a: seen.update(c_stride=a[8], k_stride=a[10], T=a[15]))
    kv = torch.zeros(576, 1, dtype=torch.bfloat16).t()
    assert kv.shape == (1, 576) and kv.stride(0) == 1
    session.append_normed_rows(None, state(), kv, torch.ones(512, dtype=torch.bfloat16), None, 1e-6,
                               torch.zeros(1, dtype=torch.int64), torch.zeros(1, dtype=torch.int32))
    assert seen == dict(c_stride=576, k_stride=576, T=1)


def test_norm_rope_rows_refuses_what_it_would_misread():
    R, H, D, bf = 3, 4, 192, torch.bfloat16
    cfg = object()  # (a call that is not refused ends before it is looked at)
    good = dict(x=torch.zeros(R, H, D, dtype=bf), weight=torch.ones(D, dtype=bf),
                positions=torch.zeros(R, dtype=torch.int64), out=None)

    def call(cfg=cfg, **over):
        a = {**good, **over}
        session.norm_rope_rows(cfg, a["x"], a["weight"], 1e-6, a["positions"], a["out"])

    reaches(call)
    reaches(lambda: call(weight=None))
    reaches(lambda: call(weight=torch.ones(H, D, dtype=bf)))
    reaches(lambda: call(weight=torch.ones(D, dtype=bf).expand(H, D)))
    reaches(lambda: call(cfg=None, positions=None))
    reaches(lambda: call(x=torch.zeros(H, R, D, dtype=bf).transpose(0, 1)))
    reaches(lambda: call(out=torch.zeros(R, 2 * H, D, dtype=bf)[:, ::2]))
    refused(lambda: call(x=torch.zeros(R, H, 2 * D, dtype=bf)[..., ::2]), "adjacent")
    refused(lambda: call(x=torch.zeros(R, H, D)), "x is")
    refused(lambda: call(weight=torch.ones(2 * D, dtype=bf)[::2]), "one behind")
    refused(lambda: call(weight=torch.ones(H, 2 * D, dtype=bf)[:, ::2]), "adjacent")
    refused(lambda: call(weight=torch.ones(H, D)), "weight")
    refused(lambda: call(weight=torch.ones(1, D, dtype=bf)), "weight")
    refused(lambda: call(weight=torch.ones(D - 1, dtype=bf)), "weight")
    refused(lambda: call(weight=torch.ones(D)), "weight")
    refused(lambda: call(out=torch.zeros(R - 1, H, D, dtype=bf)), "out")
    refused(lambda: call(out=torch.zeros(R, H, D)), "out")
    refused(lambda: call(positions=torch.zeros(R, dtype=torch.int32)), "positions")
    refused(lambda: call(positions=torch.zeros(R - 1, dtype=torch.int64)), "positions")
    refused(lambda: call(positions=torch.zeros(2 * R, dtype=torch.int64)[::2]), "positions")


def test_shared_decode_refuses_less_than_its_sizes():
    """A decoder made for more sequences, queries or prefix pages than the call brings
    would read behind the tensors (and write behind out)."""
    bf = torch.bfloat16
    good = dict(st=state(), prefix=torch.zeros(1, dtype=torch.int32), q=torch.zeros(2, 1, 32, 192, dtype=bf), out=None)

    def call(dec=None, **over):
        a = {**good, **over}
        (dec or shared_decoder()).decode(None, a["st"], a["prefix"], a["q"], 0.1, a["out"])

    reaches(call)
    reaches(lambda: call(prefix=torch.zeros(3, dtype=torch.int32)))
    reaches(lambda: call(out=torch.zeros(2, 1, 32, 128, dtype=bf)))
    refused(lambda: call(prefix=torch.zeros(0, dtype=torch.int32)), "prefix_table")
    refused(lambda: call(prefix=torch.zeros(1, dtype=torch.int64)), "prefix_table")
    refused(lambda: call(shared_decoder(prefix_pages=2)), "prefix_table")
    refused(lambda: call(prefix=torch.zeros(4, dtype=torch.int32)[::2], dec=shared_decoder(prefix_pages=2)), "prefix")
    refused(lambda: call(q=torch.zeros(1, 1, 32, 192, dtype=bf)), "q must")
    refused(lambda: call(q=torch.zeros(2, 1, 32, 192)), "q must")
    refused(lambda: call(q=torch.zeros(2, 1, 192, 32, dtype=bf).transpose(2, 3)), "q must")
    refused(lambda: call(shared_decoder(q_len=2)), "q must")
    refused(lambda: call(out=torch.zeros(1, 1, 32, 128, dtype=bf)), "out must")
    refused(lambda: call(st=state(batch=1)), "sequences")


def test_read_back_refuses_lengths_outside_the_table():
    st = state("q8")  # two sequences of up to 256 tokens
    reaches(lambda: session.read_back_q8(st, [256, 3]))
    reaches(lambda: session.read_back_q8(st, [1]))
    for bad in ([257, 3], [3, 300], [1, 2, 3], [-1, 4]):
        refused(lambda: session.read_back_q8(st, bad), "block table")
