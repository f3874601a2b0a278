"""Calls on a stream that is not the current one: where the memory of their results comes
from, and when it may be handed on.

The allocator keeps a pool per stream and orders reuse by that stream alone. A result that a
call on stream s writes has to come from s's pool: from the current stream's, it could be
memory that a kernel there still uses, or be handed out again there while s still writes it.
And the caller, who works with the result on the current stream, may drop it while that work
is under way: the memory is not handed on before it is done. Both are read off the
allocator's own record; no race is run.
"""
import pytest
import torch

import combine_topk_ids_expert_gb300 as ep
from test_expert_ffn_gpu import Case
from test_expert_w4_gpu import weights

pytestmark = pytest.mark.gpu


def pool_of(t):
    """The stream whose pool t's memory belongs to."""
    p = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= p < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


def block_states(places):
    """The allocator's words for the blocks at these addresses, from one look at its record."""
    found = dict.fromkeys(places, "gone")
    for seg in torch.cuda.memory_snapshot():
        at = seg["address"]
        for b in seg["blocks"]:
            for p in places:
                if at <= p < at + b["size"]:
                    found[p] = b["state"]
            at += b["size"]
    return found


def setup():
    c = Case(90, 64, 4, 2, 2, D=128)
    c.sc = torch.rand((64, 2), device="cuda", generator=c.gen)
    c.x = c.randn(64, 128)
    c.buf.dispatch(c.x, c.sc, c.ids, 64)
    c.rows_in, c.weights_in = c.recv(128), torch.ones(c.rows, device="cuda")
    c.wgu, c.wd = c.randn(4, 256, 128), c.randn(4, 128, 128)
    c.gate_up, c.h = c.recv(256), c.recv(128)
    c.w4gu, c.w4d = weights(c, 256, 128, 64, True, "bf16"), weights(c, 128, 128, 32, False, "f32")
    torch.cuda.synchronize()
    return c


CALLS = {
    "combine": lambda c, s: c.buf.combine(c.rows_in, c.sc, stream=s),
    "combine_backward": lambda c, s: c.buf.combine_backward(c.x, c.rows_in, c.sc, stream=s),
    "dispatch_backward": lambda c, s: c.buf.dispatch_backward(
        c.rows_in, 64, c.weights_in, stream=s),
    "expert_gemm": lambda c, s: c.buf.expert_gemm(c.rows_in, c.wd, stream=s),
    "expert_glu": lambda c, s: c.buf.expert_glu(c.rows_in, c.wgu, stream=s),
    "expert_ffn": lambda c, s: c.buf.expert_ffn(c.rows_in, c.wgu, c.wd, stream=s),
    "expert_ffn_saving": lambda c, s: c.buf.expert_ffn(c.rows_in, c.wgu, c.wd, save=True, stream=s),
    "expert_glu_backward": lambda c, s: c.buf.expert_glu_backward(c.h, c.wd, c.gate_up, stream=s),
    "expert_gemm_backward": lambda c, s: c.buf.expert_gemm_backward(c.h, c.rows_in, c.wd, stream=s),
    "expert_ffn_backward": lambda c, s: c.buf.expert_ffn_backward(
        c.h, c.rows_in, c.wgu, c.wd, c.gate_up, c.h, stream=s),
    "expert_gemv_w4": lambda c, s: c.buf.expert_gemv_w4(c.rows_in, c.w4d, stream=s),
    "expert_glu_w4": lambda c, s: c.buf.expert_glu_w4(c.rows_in, c.w4gu, stream=s),
    "expert_ffn_w4": lambda c, s: c.buf.expert_ffn_w4(c.rows_in, c.w4gu, c.w4d, stream=s),
}


def results(name, c, s):
    got = CALLS[name](c, s)
    return list(got) if isinstance(got, tuple) else [got]


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_results_come_from_the_launching_streams_pool(name, handle):
    c, s = setup(), torch.cuda.Stream()
    here = results(name, c, None)
    torch.cuda.synchronize()
    there = results(name, c, s.cuda_stream if handle else s)
    torch.cuda.synchronize()
    mine = torch.cuda.current_stream().cuda_stream
    for a, b in zip(here, there):
        assert pool_of(a) == mine and pool_of(b) == s.cuda_stream
    c.done()


def test_expanded_rows_come_from_the_launching_streams_pool():
    c, s = setup(), torch.cuda.Stream()
    c.buf.dispatch_dedup(c.x, c.sc, c.ids, 64)
    torch.cuda.synchronize()
    y = c.buf.dedup_expand(c.ids, stream=s)
    torch.cuda.synchronize()
    assert pool_of(y) == s.cuda_stream
    c.done()


@pytest.mark.parametrize("name", ["combine", "expert_ffn_saving", "expert_ffn_backward",
                                  "expert_ffn_w4"])
def test_dropped_results_wait_for_the_current_stream(name):
    c, s = setup(), torch.cuda.Stream()
    got = results(name, c, s)
    torch.cuda.synchronize()
    places = [t.data_ptr() for t in got]
    torch.cuda._sleep(400_000_000)   # about a fifth of a second of the current stream's time
    del got
    states = block_states(places)
    busy = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert busy, "the current stream was done too early to tell"
    # in use no more, and not free yet
    assert all(t.startswith("active_") and t.endswith("_free") for t in states.values()), states
    c.done()


def test_scratch_rows_come_from_the_launching_streams_pool(monkeypatch):
    c, s = setup(), torch.cuda.Stream()
    taken = []
    keep = ep.Buffer._empty

    def noted(self, shape, dtype, stream, kept=True):
        t = keep(self, shape, dtype, stream, kept)
        taken.append(t)
        return t

    monkeypatch.setattr(ep.Buffer, "_empty", noted)
    for name in ("expert_ffn", "expert_ffn_backward", "expert_ffn_w4"):
        results(name, c, s)
    torch.cuda.synchronize()
    assert len(taken) == 2 + 4 + 2
    assert {pool_of(t) for t in taken} == {s.cuda_stream}
    c.done()
