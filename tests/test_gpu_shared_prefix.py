"""GPU parity of mla_shared_prefix_attention against attention in 64 bits over each sequence's whole
table, at the sizes where packed rows, tiles, pages and parts end unevenly.

Bounds, for o = sum_j p_j v_j / l with u half a step of the element type (bf16 2^-8, fp16 2^-11):
the weights are rounded to the element type, at most u sum_j p_j |v_j|; o is rounded once, u |o|. A
score's fp32 sum of D products in steps of 16 is off by at most 2^-18 sum_d |q_d k_d| scale =: e
(36 steps and a join, each below 2^-23 of the magnitude, with room), which moves lse by e and a
weight by a factor of 1 +- 2 e. exp2 and the sums add less than 2^-17 of each. The fp32 lse has no
other error.
"""
import numpy as np
import pytest
import torch

import mla_latent_kv_42_b200 as M
from mla_latent_kv_42_b200 import build, synth

pytestmark = pytest.mark.gpu

P, R = synth.PRODUCTION, synth.RUNNING
GENERIC = R.with_(d_c=256, d_rope=32, page_size=32, n_heads=4)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    M.load_library()
    M.read_device_status()


class Case:
    """Sequences of ``lens`` tokens, those of at least ``shared`` pages behind the same pages; slots
    that hold no token of theirs are NaN."""

    def __init__(self, d, lens, shared, seed=0, scale=2.0, spare=1):
        self.d, self.lens_np, self.n_shared = d, np.asarray(lens), shared
        rng = np.random.default_rng(seed)
        page = d.page_size
        used = -(-self.lens_np // page)
        width = max(int(used.max()), shared) + spare
        uses = self.lens_np >= shared * page
        own = np.where(uses, used - shared, used).clip(0)
        ids = rng.permutation(shared + int(own.sum()) + 1)  # one page of nobody
        self.shared_np = ids[:shared].astype(np.int32)
        table = np.full((len(lens), width), -1, dtype=np.int32)
        at = shared
        for b, n in enumerate(own):
            f = shared if uses[b] else 0
            table[b, :f] = self.shared_np[:f]
            table[b, f:f + n] = ids[at:at + n]
            at += n
        e = synth.storage_dtype(d)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = torch.full((len(ids), page, d.D), float("nan"), device="cuda", dtype=e)
        for b, n in enumerate(self.lens_np):
            for j in range(used[b]):
                k = min(page, int(n) - j * page)
                if b == 0 or j >= shared or not uses[b] or not uses[:b].any():
                    self.pool[table[b, j], :k] = (0.43 * torch.randn((k, d.D), device="cuda", generator=g)).to(e)
        self.q = (scale * torch.randn((len(lens), d.n_heads, d.D), device="cuda", generator=g)).to(e)
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
        self.table, self.lens, self.shared = i32(table), i32(lens), i32(self.shared_np)
        self.longest = int(self.lens_np.max())

    def run(self, **kw):
        return M.shared_prefix_attention(self.d, self.q, self.pool, self.table, self.lens,
                                         kw.pop("longest", self.longest), self.shared, **kw)

    def check(self, o, lse, skip=(), exact_lse=True):
        d = self.d
        u = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[d.dtype]
        scale = (d.d_head + d.d_rope) ** -0.5
        for b, n in enumerate(self.lens_np):
            if b in skip:
                continue
            rows = self.pool[self.table[b, :-(-int(n) // d.page_size)].long()].reshape(-1, d.D)[:n].double()
            q = self.q[b].double()
            s = q @ rows.T * scale
            ref_l = s.logsumexp(1)
            p = (s - ref_l[:, None]).exp()
            v = rows[:, :d.d_c]
            ref, mag = p @ v, p @ v.abs()
            err = (q.abs() @ rows.abs().T * scale).amax(1) * 2.0 ** -18 + 2.0 ** -17
            tol = u * mag + u * ref.abs() + 2 * err[:, None] * mag + 2.0 ** -24
            off = (o[b].double() - ref).abs()
            assert bool((off <= tol).all()), (b, n, float((off / tol).max()))
            if lse is not None:
                slack = err + (0 if exact_lse else u)
                assert bool(((lse[b].double() - ref_l).abs() <= slack).all()), (b, n)


def batch(B, shared_len, suffixes, seed=0):
    return shared_len + np.asarray([suffixes[i % len(suffixes)] for i in range(B)])


EDGES = [1, 0, 64, 63, 65, 128, 129, 300, 2]


@pytest.mark.parametrize("heads,B,shared,dtype", [
    (16, 4, 8, "bf16"), (16, 9, 1, "fp16"), (16, 64, 3, "bf16"), (1, 7, 2, "bf16"), (1, 300, 2, "bf16"),
    (5, 27, 9, "bf16"), (33, 5, 2, "fp16"), (64, 2, 5, "bf16"), (64, 23, 4, "fp16"), (65, 11, 3, "bf16"),
    (96, 9, 2, "bf16"), (127, 130, 1, "bf16"), (128, 9, 3, "bf16"), (128, 1, 4, "fp16"), (16, 1, 4, "bf16"),
    (32, 40, 65, "bf16"), (16, 5, 0, "bf16"), (128, 4, 0, "bf16"),
    # packed rows whose last tile is short, sequences that straddle tiles, fewer places than SM pairs
    (33, 40, 9, "bf16"), (64, 40, 17, "fp16"), (65, 60, 33, "bf16"), (96, 64, 33, "bf16"), (100, 64, 41, "fp16"),
    (48, 30, 9, "fp16"), (16, 9, 40, "fp16"), (1, 7, 40, "bf16"), (3, 50, 201, "bf16"), (17, 33, 7, "bf16"),
])
def test_wide_rows(heads, B, shared, dtype):
    d = P.with_(n_heads=heads, dtype=dtype)
    lens = batch(B, shared * d.page_size, EDGES).clip(1)
    c = Case(d, lens, shared, seed=heads + B)
    o, lse = c.run()
    assert M.read_device_status() == 0
    c.check(o, lse)


@pytest.mark.parametrize("d,B,shared", [
    (R, 16, 64), (R, 1, 5), (R, 2, 1), (R, 3, 2), (R, 50, 7), (R, 5, 0), (R.with_(n_heads=1, dtype="fp16"), 100, 3),
    (R.with_(n_heads=16, page_size=16), 13, 11), (R.with_(n_heads=3, page_size=48), 31, 4),
    (R.with_(n_heads=16, d_c=16, d_rope=16, page_size=32), 9, 5), (R.with_(d_c=112, d_rope=80, page_size=64), 9, 3),
    (R.with_(n_heads=7, d_c=128, d_rope=64), 70, 33),
])
def test_narrow_rows(d, B, shared):
    lens = batch(B, shared * d.page_size, EDGES).clip(1)
    c = Case(d, lens, shared, seed=B)
    o, lse = c.run()
    assert M.read_device_status() == 0
    c.check(o, lse)


def test_other_shapes_run_as_decode():
    lens = batch(6, 3 * GENERIC.page_size, EDGES).clip(1)
    c = Case(GENERIC, lens, 3, seed=8)
    o, lse = c.run()
    assert M.read_device_status() == 0
    c.check(o, lse, exact_lse=False)


@pytest.mark.parametrize("d", [P.with_(n_heads=16), R, P], ids=["h16", "narrow", "h128"])
def test_idle_rows_and_peaked_softmax(d):
    """Rows of a padded batch (one token, or a few below the prefix) attend to their own pages alone;
    scores of hundreds make single weights decide."""
    lens = batch(20, 4 * d.page_size, [1, 70, 200])
    lens[[0, 3, 19]] = [1, 1, 4 * d.page_size - 1]
    c = Case(d, lens, 4, seed=3, scale=60.0)
    o, lse = c.run()
    assert M.read_device_status() == 0
    c.check(o, lse)


def test_a_batch_of_idle_rows_only():
    d = P.with_(n_heads=16)
    c = Case(d, [1, 5, 64, 100], 3, seed=4)
    o, lse = c.run(longest=256)
    assert M.read_device_status() == 0
    c.check(o, lse)


@pytest.mark.parametrize("d,B", [(P.with_(n_heads=1), 5000), (R.with_(n_heads=2), 5000)], ids=["wide", "narrow"])
def test_many_sequences(d, B):
    lens = batch(B, 2 * d.page_size, [1, 0, 3, 65, 1, 1])
    c = Case(d, lens, 2, seed=5)
    o, lse = c.run()
    assert M.read_device_status() == 0
    c.check(o, lse, skip=set(range(20, B - 20)))
    ref_o, ref_l = M.decode_attention(d, c.q, c.pool, c.table, c.lens, c.longest)
    assert float((o.float() - ref_o.float()).abs().max()) < 2e-2
    assert float((lse - ref_l).abs().max()) < 2.0 ** -8


@pytest.mark.parametrize("heads,B,shared,longest", [(16, 300, 4, 0), (128, 40, 2, 40000), (16, 40, 8, 40000)])
def test_plan_as_a_kernel_of_its_own(heads, B, shared, longest):
    """Many sequences, or a bound on their lengths that allows many pages: three launches instead of two."""
    d = P.with_(n_heads=heads)
    c = Case(d, batch(B, shared * d.page_size, EDGES), shared, seed=15, spare=650 if longest else 1)
    o, lse = c.run()
    few = M.last_launch_count(M.CALL_SHARED_PREFIX_ATTENTION)
    c.check(o, lse)
    o, lse = c.run(longest=longest or c.longest)
    assert M.read_device_status() == 0
    assert M.last_launch_count(M.CALL_SHARED_PREFIX_ATTENTION) == 3 and few == (2 if longest else 3)
    c.check(o, lse)


@pytest.mark.parametrize("d", [P.with_(n_heads=16), P.with_(n_heads=48), P, R], ids=["h16", "h48", "h128", "narrow"])
def test_agrees_with_decode_and_repeats_bitwise(d):
    lens = batch(24, 40 * d.page_size, [1, 500, 64, 1000])
    c = Case(d, lens, 40, seed=6)
    o, lse = c.run()
    for _ in range(3):
        o2, lse2 = c.run()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    ref_o, ref_l = M.decode_attention(d, c.q, c.pool, c.table, c.lens, c.longest)
    assert M.read_device_status() == 0
    assert float((o.float() - ref_o.float()).abs().max()) <= 2.0 ** -6 * float(ref_o.float().abs().max())
    assert float((lse - ref_l).abs().max()) <= 2.0 ** -8


@pytest.mark.parametrize("d,shared", [(P.with_(n_heads=16), 2), (P.with_(n_heads=16), 40), (P.with_(n_heads=96), 2),
                                      (P.with_(n_heads=80), 60), (P, 2), (R, 2), (GENERIC, 2)],
                         ids=["h16", "h16-packed", "h96", "h80-packed", "h128", "narrow", "generic"])
def test_rejected_sequences(d, shared):
    """A bad length or own page rejects its sequence alone; a bad shared page every one that has it."""
    lens = batch(12, shared * d.page_size, [1, 70, 130])
    lens[5] = 3  # idle
    c = Case(d, lens, shared, seed=7)
    good_o, good_l = c.run()
    assert M.read_device_status() == 0
    lens_bad = c.lens.clone()
    lens_bad[2], lens_bad[8] = 0, c.longest + 1
    table_bad = c.table.clone()
    table_bad[4, shared] = len(c.pool)
    table_bad[7, shared] = -1
    o, lse = M.shared_prefix_attention(d, c.q, c.pool, table_bad, lens_bad, c.longest, c.shared)
    assert M.read_device_status() in (-7, -8)
    for b in range(12):
        if b in (2, 4, 7, 8):
            assert not bool(o[b].any()) and bool((lse[b] == -float("inf")).all()), b
    c.check(o, lse, skip=(2, 4, 7, 8), exact_lse=d is not GENERIC)
    shared_bad, table_bad = c.shared.clone(), c.table.clone()
    shared_bad[1] = len(c.pool) + 5
    has = [b for b in range(12) if b != 5]
    table_bad[has, 1] = len(c.pool) + 5
    o, lse = M.shared_prefix_attention(d, c.q, c.pool, table_bad, c.lens, c.longest, shared_bad)
    assert M.read_device_status() == -7
    assert not bool(o[has].any()) and bool((lse[has] == -float("inf")).all())
    c.check(o, lse, skip=has, exact_lse=d is not GENERIC)
    o, lse = c.run()
    assert M.read_device_status() == 0 and torch.equal(o, good_o) and torch.equal(lse, good_l)


@pytest.mark.parametrize("shared", [2, 30])
def test_without_lse_given_outputs_and_no_sequences(shared):
    d = P.with_(n_heads=16)
    c = Case(d, batch(5, 64 * shared, [1, 9]), shared, seed=1)
    o, lse = c.run()
    out = torch.empty_like(o)
    ws = torch.empty(M.workspace_size(d, M.CALL_SHARED_PREFIX_ATTENTION, 5, c.longest), dtype=torch.uint8,
                     device="cuda")
    ws.fill_(0xFF)  # NaN partials: nothing is read that this call did not write
    got, none = c.run(o_lat=out, want_lse=False, ws=ws)
    assert got is out and none is None and torch.equal(got, o)
    e, l = M.shared_prefix_attention(d, c.q[:0], c.pool, c.table[:0], c.lens[:0], c.longest, c.shared)
    assert e.shape == (0, 16, 512) and l.shape == (0, 16)
    assert M.last_launch_count(M.CALL_SHARED_PREFIX_ATTENTION) == 0
    assert M.read_device_status() == 0


@pytest.mark.parametrize("d", [P.with_(n_heads=16), R], ids=["h16", "narrow"])
def test_captured_and_replayed_as_lengths_grow(d):
    lens = batch(8, 24 * d.page_size, [1, 60, 126])
    c = Case(d, lens + 4, 24, seed=2)  # rows for every step below
    c.lens.copy_(torch.from_numpy(lens.astype(np.int32)))
    ws = torch.empty(M.workspace_size(d, M.CALL_SHARED_PREFIX_ATTENTION, 8, c.longest), dtype=torch.uint8,
                     device="cuda")
    o, lse = c.run(ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(o_lat=o, lse=lse, ws=ws)
    for step in range(5):
        graph.replay()
        torch.cuda.synchronize()
        c.lens_np = lens + step
        c.check(o, lse)
        c.lens += 1
    assert M.read_device_status() == 0


@pytest.mark.parametrize("d,shared", [(P.with_(n_heads=16), 30), (P.with_(n_heads=16), 2), (P, 3), (R, 5), (R, 0)],
                         ids=["h16-packed", "h16", "h128", "narrow", "narrow-alone"])
def test_not_a_number_stays_in_its_sequence(d, shared):
    """A NaN in a sequence's queries, or in one of its own cached rows, is in that sequence's output
    (its head's, or all heads') and changes no other bit."""
    c = Case(d, batch(12, shared * d.page_size, [70, 1, 200]).clip(1), shared, seed=12)
    o, lse = c.run()
    c.q[3, 1, 5] = float("nan")
    c.pool[c.table[6, (int(c.lens_np[6]) - 1) // d.page_size].long(), (int(c.lens_np[6]) - 1) % d.page_size] = float("nan")
    got_o, got_l = c.run()
    assert M.read_device_status() == 0
    same = [b for b in range(12) if b not in (3, 6)]
    assert torch.equal(got_o[same], o[same]) and torch.equal(got_l[same], lse[same])
    heads = [h for h in range(d.n_heads) if h != 1]
    assert torch.equal(got_o[3, heads], o[3, heads]) and torch.equal(got_l[3, heads], lse[3, heads])
    assert bool(got_o[3, 1].isnan().all()) and bool(got_l[3, 1].isnan())
    assert bool(got_o[6].isnan().all()) and bool(got_l[6].isnan().all())


def test_two_streams_at_once():
    cases = [Case(P.with_(n_heads=16), batch(20, 64 * 30, EDGES), 30, seed=s) for s in (1, 2)]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    wss = [torch.empty(M.workspace_size(c.d, M.CALL_SHARED_PREFIX_ATTENTION, 20, c.longest), dtype=torch.uint8,
                       device="cuda") for c in cases]
    outs = [(torch.empty_like(o), torch.empty_like(l)) for o, l in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, w, (o, l) in zip(cases, streams, wss, outs):
            c.run(o_lat=o, lse=l, ws=w, stream=s)
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)
    assert M.read_device_status() == 0


@pytest.mark.parametrize("d", [R, P.with_(n_heads=16, d_model=1024, d_cq=256)], ids=["running", "h16"])
def test_layer_step_behind_a_shared_prefix(d):
    """A whole layer step with shared pages: the step without them to the rounding of o_lat (half a step
    on either side, then a product over n_h d_h values of it), its appended rows bit for bit."""
    from mla_latent_kv_42_b200 import LayerState
    lens = batch(24, 20 * d.page_size, [1, 70, 64])
    c = Case(d, lens, 20, seed=14)
    g = torch.Generator(device="cuda").manual_seed(1)
    e = synth.storage_dtype(d)
    w = {k: (0.02 * torch.randn(s, device="cuda", generator=g)).to(e) for k, s in synth._weight_shapes(d).items()}
    h = torch.randn((24, d.d_model), device="cuda", generator=g).to(e)
    seq = torch.arange(24, dtype=torch.int32, device="cuda")
    other = c.pool.clone()
    ws = torch.empty(M.step_workspace_bytes(d, 24, c.longest, shared=True), dtype=torch.uint8, device="cuda")
    u, q, o, lse = M.layer_step(LayerState(d, w, c.pool, c.table), h, c.lens - 1, seq, c.lens, c.longest, ws=ws,
                                shared_pages=c.shared)
    u2, q2, o2, lse2 = M.layer_step(LayerState(d, w, other, c.table), h, c.lens - 1, seq, c.lens, c.longest)
    assert M.read_device_status() == 0
    assert torch.equal(c.pool.view(torch.int16), other.view(torch.int16)) and torch.equal(q, q2)
    assert float((o.float() - o2.float()).abs().max()) <= 2.0 ** -6 * float(o2.float().abs().max())
    assert float((u.float() - u2.float()).abs().max()) <= 2.0 ** -5 * float(u2.float().abs().max())
    assert float((lse - lse2).abs().max()) <= 2.0 ** -8


def test_together_fp8_prefix_written_read_back_and_shared():
    """The calls as they are used: a prefix normalised, rotated and quantised into the FP8 cache, read
    back into element-type pages, the sequences' own rows written beside them, and one attention
    over both."""
    d = P.with_(n_heads=16)
    page, shared, B = d.page_size, 12, 9
    g = torch.Generator(device="cuda").manual_seed(0)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    gain = (1 + 0.1 * torch.randn(d.d_c, device="cuda", generator=g)).bfloat16()
    n = shared * page
    x = torch.randn((n, d.D), device="cuda", generator=g).bfloat16()
    cold = torch.empty((shared, M.fp8_page_bytes(d)), dtype=torch.uint8, device="cuda")
    pos, zero, cold_table = i32(list(range(n))), i32([0] * n), i32([[4, 2, 0, 11, 3, 7, 5, 10, 1, 6, 9, 8]])
    M.norm_append_kv_fp8(d, x, zero, pos, cold_table, cold, gain_c=gain)
    lens = batch(B, n, [1, 64, 70])
    c = Case(d, lens, shared, seed=11)
    pages = c.pool[:0].new_empty((shared, page, d.D))
    M.read_kv_fp8(d, cold, zero, pos, cold_table, out=pages.view(n, d.D))
    c.pool[c.shared.long()] = pages
    # each sequence's last token arrives now
    new = torch.randn((B, d.D), device="cuda", generator=g).bfloat16()
    M.norm_append_kv(d, new, i32(list(range(B))), c.lens - 1, c.table, c.pool, gain_c=gain)
    o, lse = c.run()
    assert M.read_device_status() == 0
    c.check(o, lse)
    # what the prefix pages hold is the definition to an e4m3 step
    xr = x.double()
    ref = xr[:, :d.d_c] / (xr[:, :d.d_c].square().mean(1, keepdim=True) + 1e-6).sqrt() * gain.double()
    off = (pages.view(n, d.D)[:, :d.d_c].double() - ref).abs()
    peak = ref.abs().amax(1, keepdim=True)
    assert bool((off <= (2.0 ** -4 + 2.0 ** -7) * ref.abs() + peak * 2.0 ** -10 / 448 + 1e-5).all())
