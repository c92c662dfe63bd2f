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
