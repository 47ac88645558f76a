"""Calls on a stream of their own, with outputs and workspaces that they allocate themselves: those come from
that stream's memory, since what the current stream has freed may still be in use by what it has queued."""
import numpy as np
import pytest
import torch

import mla_latent_kv_42_b200 as M
from mla_latent_kv_42_b200 import build, synth

pytestmark = pytest.mark.gpu

P = synth.PRODUCTION.with_(d_model=1024, d_cq=256, n_heads=80)
H20 = P.with_(n_heads=20)
R = synth.RUNNING


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    M.load_library()
    M.read_device_status()


class State:
    """Inputs of every call: B sequences of ``n`` tokens, the last of which is new."""

    def __init__(self, d, seed, B=20, n=900):
        g = torch.Generator(device="cuda").manual_seed(seed)
        e = synth.storage_dtype(d)
        rnd = lambda *shape, std=1.0: (std * torch.randn(shape, device="cuda", generator=g)).to(e)
        pages = -(-n // d.page_size)
        self.d, self.n = d, n
        self.pool = rnd(B * pages, d.page_size, d.D, std=0.43)
        self.pool8 = torch.zeros((B * pages, M.fp8_page_bytes(d)), dtype=torch.uint8, device="cuda")
        self.w = {k: rnd(*s, std=0.02) for k, s in synth._weight_shapes(d).items()}
        self.h, self.q = rnd(B, d.d_model), rnd(B, d.n_heads, d.D, std=2.0)
        self.o, self.x = rnd(B, d.n_heads, d.d_c), rnd(B, d.D)
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
        table = np.arange(B * pages).reshape(B, pages)
        table[:, :10] = np.arange(10)
        self.table, self.shared = i32(table), i32(np.arange(10))
        self.seq, self.lens, self.pos = i32(np.arange(B)), i32(np.full(B, n)), i32(np.full(B, n - 1))
        self.all_seq = self.seq.repeat_interleave(n)
        self.all_pos = i32(np.tile(np.arange(n), B))
        M.norm_append_kv_fp8(d, self.pool.view(-1, d.D)[:B * pages * d.page_size].contiguous(),
                             i32(np.arange(B * pages * d.page_size) // d.page_size),
                             i32(np.arange(B * pages * d.page_size) % d.page_size), i32(np.arange(B * pages)[:, None]),
                             self.pool8)


CALLS = {
    "append_kv": (H20, lambda s, **k: M.append_kv(s.d, s.h, s.w["w_dkv_kr"], s.seq, s.pos, s.table, s.pool, **k)),
    "append_kv_fp8": (P, lambda s, **k: M.append_kv_fp8(s.d, s.h, s.w["w_dkv_kr"], s.seq, s.pos, s.table, s.pool8, **k)),
    "absorb_query": (H20, lambda s, **k: M.absorb_query(s.d, s.h, s.w["w_dq"], s.w["w_uq_qr"], s.w["w_uk"], s.pos, **k)),
    "decode": (P, lambda s, **k: M.decode_attention(s.d, s.q, s.pool, s.table, s.lens, s.n, **k)),
    "decode_narrow": (R, lambda s, **k: M.decode_attention(s.d, s.q, s.pool, s.table, s.lens, s.n, **k)),
    "decode_fp8": (P, lambda s, **k: M.decode_attention_fp8(s.d, s.q, s.pool8, s.table, s.lens, s.n, **k)),
    "prefill": (P, lambda s, **k: M.prefill_attention(s.d, s.q, s.pool, s.table, s.seq, s.pos, s.n, **k)),
    "out_proj": (H20, lambda s, **k: M.out_proj(s.d, s.o, s.w["w_uv"], s.w["w_o"], **k)),
    "read_kv": (P, lambda s, **k: M.read_kv(s.d, s.pool, s.all_seq, s.all_pos, s.table, **k)),
    "read_kv_fp8": (P, lambda s, **k: M.read_kv_fp8(s.d, s.pool8, s.all_seq, s.all_pos, s.table, **k)),
    "shared": (H20, lambda s, **k: M.shared_prefix_attention(s.d, s.q, s.pool, s.table, s.lens, s.n, s.shared, **k)),
    "shared_narrow": (R, lambda s, **k: M.shared_prefix_attention(s.d, s.q, s.pool, s.table, s.lens, s.n, s.shared, **k)),
    "layer_step": (H20, lambda s, **k: M.layer_step(M.LayerState(s.d, s.w, s.pool, s.table), s.h, s.pos, s.seq, s.lens,
                                                    s.n, shared_pages=s.shared, **k)),
    "layer_step_small": (R, lambda s, **k: M.layer_step_small(M.LayerState(s.d, s.w, s.pool, s.table), s.h, s.lens, s.n,
                                                              **k)),
}


def tensors(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


@pytest.mark.parametrize("name", list(CALLS))
def test_current_and_side_stream_in_turn(name):
    """Ten calls on the current stream between ten on another, each with tensors of its own: every
    result is that of the call alone, also where the outputs of the calls before have been dropped."""
    d, call = CALLS[name]
    here, there = State(d, 1), State(d, 2)
    want = [[t.clone() for t in tensors(call(s))] for s in (here, there)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        a = tensors(call(here))
        b = tensors(call(there, stream=side))
    torch.cuda.synchronize()
    for got, ref in zip((a, b), want):
        assert len(got) == len(ref) and all(torch.equal(x, y) for x, y in zip(got, ref))
    assert M.read_device_status() == 0


@pytest.mark.parametrize("name", ["read_kv", "shared", "decode"])
def test_outputs_come_from_the_streams_own_memory(name):
    """Nothing that the current stream has freed is handed to a call on another stream."""
    d, call = CALLS[name]
    s, side = State(d, 3), torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [[torch.empty_like(t) for t in tensors(call(s))] for _ in range(4)]
    ranges = [(t.data_ptr(), t.data_ptr() + t.nbytes) for ts in freed for t in ts]
    del freed
    got = tensors(call(s, stream=side))
    side.synchronize()
    for t in got:
        assert all(t.data_ptr() >= hi or t.data_ptr() + t.nbytes <= lo for lo, hi in ranges)
    assert M.read_device_status() == 0


def test_given_tensors_are_used_on_a_side_stream_too():
    s, side = State(H20, 4), torch.cuda.Stream()
    want = M.shared_prefix_attention(s.d, s.q, s.pool, s.table, s.lens, s.n, s.shared)
    o, lse = (torch.empty_like(t) for t in want)
    side.wait_stream(torch.cuda.current_stream())
    got = M.shared_prefix_attention(s.d, s.q, s.pool, s.table, s.lens, s.n, s.shared, o_lat=o, lse=lse, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got[0] is o and torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("name", ["read_kv", "shared", "shared_narrow", "absorb_query"])
def test_captured_on_a_forked_stream(name):
    """A call on a stream that a capture forks to, with tensors of its own, replayed with other inputs."""
    d, call = CALLS[name]
    s, other, side = State(d, 5), State(d, 6), torch.cuda.Stream()
    call(s)
    want = [t.clone() for t in tensors(call(other))]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(2):  # the first one's tensors are freed within the capture
            got = tensors(call(s, stream=side))
        torch.cuda.current_stream().wait_stream(side)
    for a, b in ((s.pool, other.pool), (s.q, other.q), (s.h, other.h), *((s.w[k], other.w[k]) for k in s.w)):
        a.copy_(b)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert M.read_device_status() == 0
