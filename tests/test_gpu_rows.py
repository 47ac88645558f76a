"""GPU parity of the row calls (mla_norm_append_kv, mla_norm_append_kv_fp8, mla_read_kv,
mla_read_kv_fp8) against their definition in 64 bits.

Bounds. A 16-bit row value is rounded once from fp32: half a step, ``finfo.eps / 2`` of the value
(2^-25 for an fp16 subnormal). Before that, in fp32 units of 2^-24: the sum of squares adds 24
products on a lane and five levels of a tree, rsqrt and the three products add a few more, 40 in
all, halved by the root; a rotation adds the rounded cosine and sine (2 units each of a turn's
rest rounded at 2^-26 turns: 2 pi 2^-26 < 2 units) to its two products. 64 units of |value| and, for
a rotated pair, of |x0| + |x1|, cover both. An e4m3 byte is off by half a step, 2^-4 of the value,
or half the smallest subnormal, 2^-10, of value / scale.
"""
import dataclasses

import numpy as np
import pytest
import torch

import mla_latent_kv_42_b200 as M
import oracle as O
from mla_latent_kv_42_b200 import build, synth

pytestmark = pytest.mark.gpu

F32 = 64 * 2.0 ** -24
TINY = synth.RUNNING.with_(d_c=8, d_rope=8, page_size=65536)
ODD = synth.RUNNING.with_(d_c=248, d_rope=24, page_size=7)
WIDE_ROPE = synth.RUNNING.with_(d_c=8, d_rope=568, page_size=5)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    M.load_library()
    M.read_device_status()


def half_step(d):
    return {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[d.dtype]


def fp8_views(pool, d):
    n = d.page_size * d.D
    return (pool[:, :n].unflatten(1, (d.page_size, d.D)),
            pool[:, n:].contiguous().view(torch.float32).unflatten(1, (d.page_size, 2)))


def make_pool(d, pages, fp8, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if not fp8:
        return torch.randn((pages, d.page_size, d.D), device="cuda", generator=g).to(synth.storage_dtype(d))
    return torch.randint(0, 256, (pages, M.fp8_page_bytes(d)), device="cuda", dtype=torch.uint8, generator=g)


def tokens(d, T, seqs, far, seed):
    """T tokens at distinct positions of ``seqs`` sequences up to ``far``, in shuffled order, and a
    table of shuffled pages for the positions that are used."""
    rng = np.random.default_rng(seed)
    seq = rng.integers(0, seqs, T)
    pos = np.empty(T, dtype=np.int64)
    for s in range(seqs):
        at = np.flatnonzero(seq == s)
        pos[at] = far - rng.permutation(max(len(at), min(far + 1, 3 * len(at))))[:len(at)]
    assert pos.min(initial=0) >= 0
    used = sorted({(int(s), int(p) // d.page_size) for s, p in zip(seq, pos)})
    table = np.full((seqs, far // d.page_size + 1), -1, dtype=np.int32)
    ids = rng.permutation(len(used) + 2)
    for i, (s, p) in enumerate(used):
        table[s, p] = ids[i]
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()
    return i32(seq), i32(pos), i32(table), len(used) + 2


def reference_rows(d, x, pos, gain_c, gain_r, eps):
    """(rows in float64, magnitude that the fp32 error is relative to)."""
    x = x.double().cpu().numpy()
    c, k = x[:, :d.d_c], x[:, d.d_c:]
    if gain_c is not None:
        c = c / np.sqrt((c * c).mean(1, keepdims=True) + eps) * gain_c.double().cpu().numpy()
    if gain_r is not None:
        k = k / np.sqrt((k * k).mean(1, keepdims=True) + eps) * gain_r.double().cpu().numpy()
    theta = d.rope_inv_freq if d.rope_inv_freq is not None else d.rope_base ** (-2.0 * np.arange(d.d_rope // 2) / d.d_rope)
    ang = pos.cpu().numpy().astype(np.float64)[:, None] * np.asarray(theta)
    z = (k[:, 0::2] + 1j * k[:, 1::2]) * np.exp(1j * ang)
    rot = np.stack([z.real, z.imag], 2).reshape(k.shape)
    mag = np.repeat(np.abs(k[:, 0::2]) + np.abs(k[:, 1::2]), 2, axis=1)
    return np.concatenate([c, rot], 1), np.concatenate([np.abs(c), mag], 1)


def slots_of(d, seq, pos, table):
    s, p, t = seq.long(), pos.long(), table.long()
    return t[s, p // d.page_size], p % d.page_size


def gains_of(d, gains, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    one = lambda n: (1 + 0.2 * torch.randn(n, device="cuda", generator=g)).to(synth.storage_dtype(d))
    return (one(d.d_c) if "c" in gains else None), (one(d.d_rope) if "r" in gains else None)


CASES = [
    # dims, tokens, sequences, farthest position, gains, extra columns of the row stride
    (synth.PRODUCTION, 1, 1, 0, "c", 0),
    (synth.PRODUCTION, 77, 5, 131071, "cr", 8),
    (synth.PRODUCTION.with_(dtype="fp16"), 130, 64, 4096, "", 1536),
    (synth.RUNNING, 9, 1, 300, "r", 24),
    (synth.RUNNING.with_(dtype="fp16", page_size=16), 20000, 16, 9000, "c", 0),
    (ODD, 33, 3, 40, "cr", 0),
    (WIDE_ROPE, 12, 2, 1000, "cr", 0),
    (TINY, 50, 2, 2 ** 31 - 1, "", 0),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["elem", "fp8"])
@pytest.mark.parametrize("d,T,seqs,far,gains,extra", CASES)
def test_norm_append_against_definition(d, T, seqs, far, gains, extra, fp8):
    seq, pos, table, pages = tokens(d, T, seqs, far, seed=T)
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, d.D + extra), device="cuda", generator=g).to(synth.storage_dtype(d))[:, :d.D]
    gc, gr = gains_of(d, gains)
    pool = make_pool(d, pages, fp8)
    before = pool.clone()
    call = M.norm_append_kv_fp8 if fp8 else M.norm_append_kv
    assert call(d, x, seq, pos, table, pool, gain_c=gc, gain_r=gr, eps=1e-5) is pool
    assert M.read_device_status() == 0
    ref, mag = reference_rows(d, x, pos, gc, gr, 1e-5)
    pg, row = slots_of(d, seq, pos, table)
    if not fp8:
        got = pool[pg, row].double().cpu().numpy()
        tol = half_step(d) * np.abs(ref) + F32 * mag + 2.0 ** -25
        assert (np.abs(got - ref) <= tol).all(), np.max(np.abs(got - ref) / tol)
        pool[pg, row] = before[pg, row]
        assert torch.equal(pool.view(torch.int16), before.view(torch.int16))  # other slots as they were
        return
    codes, scales = fp8_views(pool, d)
    got_s = scales[pg, row].double().cpu().numpy()
    parts = [slice(0, d.d_c), slice(d.d_c, d.D)]
    peak = np.stack([np.abs(ref[:, p]).max(1) for p in parts], 1)
    near = np.stack([mag[:, p].max(1) for p in parts], 1)
    assert (np.abs(got_s * 448 - peak) <= (F32 + 2.0 ** -23) * near).all()
    got = codes[pg, row].view(torch.float8_e4m3fn).double().cpu().numpy()
    for i, p in enumerate(parts):
        want = ref[:, p] / got_s[:, i:i + 1]
        tol = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 + (F32 + 2.0 ** -23) * mag[:, p] / got_s[:, i:i + 1]
        assert (np.abs(got[:, p] - want) <= tol).all()
    # other slots as they were
    old_codes, old_scales = fp8_views(before, d)
    codes, scales = codes.clone(), scales.clone()
    codes[pg, row], scales[pg, row] = old_codes[pg, row], old_scales[pg, row]
    assert torch.equal(codes, old_codes) and torch.equal(scales.view(torch.int32), old_scales.view(torch.int32))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_fp8_bytes_equal_the_oracle_without_norm_at_position_zero(dtype):
    """No gains and position 0 (no rotation): the values are the given ones, so bytes and scales are
    the oracle's bit for bit, an all-zero part among them."""
    d = synth.PRODUCTION.with_(dtype=dtype)
    T = 40
    x = synth.to_storage(np.random.default_rng(5).standard_normal((T, d.D)).astype(np.float32), d)
    x[3, :d.d_c] = 0
    x[4, d.d_c:] = 0
    x[5] = 0
    seq = torch.arange(T, dtype=torch.int32, device="cuda")
    table = torch.randperm(T, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()[:, None].contiguous()
    pool = make_pool(d, T, True)
    M.norm_append_kv_fp8(d, x.cuda(), seq, torch.zeros_like(seq), table, pool)
    vals, sc = O.quantize_rows_fp8(x.double().numpy(), d.d_c)
    codes, scales = fp8_views(pool, d)
    got = codes[table[:, 0].long(), 0].view(torch.float8_e4m3fn).double().cpu().numpy()
    np.testing.assert_array_equal(got, vals)
    np.testing.assert_array_equal(scales[table[:, 0].long(), 0].cpu().numpy(), sc.astype(np.float32))


def test_norm_append_agrees_with_append_kv():
    """Rows that mla_append_kv computes from h = one-hot columns are the weight's columns, exact: the
    row call on those columns writes the same pool to half a step of the rotation's rounding."""
    w = synth.workload("production_b64_n4096_bf16")
    d = w.dims
    W = synth.weights(w)["w_dkv_kr"].cuda()
    T = 9
    cols = torch.arange(T) * 31
    h = torch.zeros((T, d.d_model), dtype=torch.bfloat16, device="cuda")
    h[torch.arange(T), cols] = 1
    seq, pos, table, pages = tokens(d, T, 2, 500, seed=2)
    a, b = make_pool(d, pages, False), make_pool(d, pages, False)
    M.append_kv(d, h, W, seq, pos, table, a)
    M.norm_append_kv(d, W[:, cols].T.contiguous(), seq, pos, table, b)
    assert M.read_device_status() == 0
    pg, row = slots_of(d, seq, pos, table)
    assert torch.equal(a[pg, row][:, :d.d_c], b[pg, row][:, :d.d_c])
    diff = (a[pg, row].double() - b[pg, row].double()).abs()
    assert bool((diff <= 2 * 2.0 ** -8 * b[pg, row].double().abs() + 1e-6).all())


def test_rope_table_and_zero_rows():
    d = synth.PRODUCTION
    d = dataclasses.replace(d, rope_inv_freq=tuple(0.5 ** k for k in range(d.d_rope // 2)))
    T = 6
    seq, pos, table, pages = tokens(d, T, 1, 70000, seed=9)
    x = torch.randn((T, d.D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(9)).bfloat16()
    x[2] = 0
    gc, gr = gains_of(d, "cr")
    pool = make_pool(d, pages, False)
    M.norm_append_kv(d, x, seq, pos, table, pool, gain_c=gc, gain_r=gr)
    ref, mag = reference_rows(d, x, pos, gc, gr, 1e-6)
    pg, row = slots_of(d, seq, pos, table)
    got = pool[pg, row].double().cpu().numpy()
    assert (np.abs(got - ref) <= half_step(d) * np.abs(ref) + F32 * mag).all()
    assert not got[2].any()


def test_fp8_not_finite_values_stay_in_their_row():
    d = synth.PRODUCTION
    x = torch.ones((3, d.D), dtype=torch.bfloat16, device="cuda")
    x[0, 7] = float("nan")
    x[1, 9] = float("inf")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    pool = make_pool(d, 1, True)
    M.norm_append_kv_fp8(d, x, i32(0, 0, 0), i32(0, 1, 2), i32(0)[None], pool)
    got = M.read_kv_fp8(d, pool, i32(0, 0, 0), i32(0, 1, 2), i32(0)[None]).float()
    assert M.read_device_status() == 0
    assert got[0, 7].isnan() and bool((got[0, :7] == 1).all()) and bool((got[0, 8:d.d_c] == 1).all())
    assert bool(got[1, :d.d_c].isnan().all())
    assert bool(got[2, :d.d_c].eq(1).all())


@pytest.mark.parametrize("fp8", [False, True], ids=["elem", "fp8"])
@pytest.mark.parametrize("d,T", [(synth.PRODUCTION, 1), (synth.PRODUCTION, 1021), (synth.RUNNING, 6),
                                 (synth.RUNNING.with_(dtype="fp16", page_size=16), 50003), (ODD, 35), (WIDE_ROPE, 10)])
def test_read_is_exact(d, T, fp8):
    """16-bit rows come back bit for bit; e4m3 rows as scale times value in fp32, rounded once (the
    product of a 4-bit and a 24-bit value is rounded in fp32 first on both sides). Tokens in any
    order and more than once, into strided rows whose other columns stay."""
    seq, pos, table, pages = tokens(d, T, min(T, 7), 3 * T + 5, seed=T)
    again = torch.randint(0, T, (T // 3,), generator=torch.Generator().manual_seed(4)).cuda()
    seq, pos = torch.cat([seq, seq[again]]), torch.cat([pos, pos[again]])
    pool = make_pool(d, pages, fp8, seed=T)
    e = synth.storage_dtype(d)
    wide = torch.full((len(seq), d.D + 16), 7.0, dtype=e, device="cuda")
    if fp8:  # any byte but NaN, scales a cache can hold
        n = d.page_size * d.D
        pool[:, :n][(pool[:, :n] & 0x7F) == 0x7F] = 0
        sc = torch.rand((pages, 2 * d.page_size), device="cuda") * 2e-2 + 1e-4
        pool[:, n:] = sc.view(torch.uint8)
    call = M.read_kv_fp8 if fp8 else M.read_kv
    out = call(d, pool, seq, pos, table, out=wide[:, 8:8 + d.D])
    fresh = call(d, pool, seq, pos, table)
    assert M.read_device_status() == 0
    pg, row = slots_of(d, seq, pos, table)
    if fp8:
        codes, scales = fp8_views(pool, d)
        s = scales[pg, row].repeat_interleave(torch.tensor([d.d_c, d.d_rope], device="cuda"), 1)
        want = (codes[pg, row].view(torch.float8_e4m3fn).float() * s).to(e)
    else:
        want = pool[pg, row]
    assert torch.equal(fresh.view(torch.int16), want.view(torch.int16))
    assert torch.equal(out.contiguous().view(torch.int16), want.view(torch.int16))
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + d.D:] == 7).all())


@pytest.mark.parametrize("fp8", [False, True], ids=["elem", "fp8"])
def test_bad_slots_are_recorded_and_the_others_done(fp8):
    d = synth.PRODUCTION
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    table = i32([[0, 1], [3, -1], [2, 99]])
    seq, pos = i32([0, -1, 3, 0, 0, 1, 2, 2]), i32([65, 0, 0, -1, 128, 64, 64, 1])
    good = [0, 7]
    x = torch.randn((8, d.D), device="cuda").bfloat16()
    pool = make_pool(d, 4, fp8)
    before = pool.clone()
    append, read = (M.norm_append_kv_fp8, M.read_kv_fp8) if fp8 else (M.norm_append_kv, M.read_kv)
    append(d, x, seq, pos, table, pool)
    assert M.read_device_status() == -7
    want = before.clone()
    append(d, x[good].contiguous(), seq[good].contiguous(), pos[good].contiguous(), table, want)
    assert M.read_device_status() == 0
    assert torch.equal(pool.view(torch.uint8), want.view(torch.uint8))
    rows = read(d, pool, seq, pos, table)
    assert M.read_device_status() == -7
    bad = [i for i in range(8) if i not in good]
    assert not bool(rows[bad].any()) and bool(rows[good].abs().sum(1).gt(0).all())


def test_slots_past_32_bits():
    """A pool of more than 2^32 bytes: the last page's rows are written and read in place."""
    d = synth.PRODUCTION
    pages = 2 ** 32 // (d.page_size * d.D * 2) + 3
    pool = torch.empty((pages, d.page_size, d.D), dtype=torch.bfloat16, device="cuda")
    pool[-1] = 0
    pool[0] = 0
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    x = torch.randn((2, d.D), device="cuda").bfloat16()
    seq, pos, table = i32([0, 0]), i32([0, 127]), i32([[0, pages - 1]])
    M.norm_append_kv(d, x, seq, pos, table, pool)
    assert torch.equal(M.read_kv(d, pool, seq, pos, table)[0, :d.d_c], x[0, :d.d_c])
    assert torch.equal(pool[-1, 63, :d.d_c], x[1, :d.d_c]) and not bool(pool[-1, :63].any())
    assert M.read_device_status() == 0


def test_no_tokens_a_side_stream_and_a_graph():
    d = synth.RUNNING
    T = 5
    seq, pos, table, pages = tokens(d, T, 2, 100, seed=1)
    x = torch.randn((T, d.D), device="cuda").bfloat16()
    pool = make_pool(d, pages, False)
    before = pool.clone()
    M.norm_append_kv(d, x[:0], seq[:0], pos[:0], table, pool)
    assert torch.equal(pool, before) and M.last_launch_count(M.CALL_NORM_APPEND_KV) == 0
    assert M.read_kv(d, pool, seq[:0], pos[:0], table).shape == (0, d.D)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty((T, d.D), dtype=torch.bfloat16, device="cuda")
    M.norm_append_kv(d, x, seq, pos, table, pool, stream=side)
    M.read_kv(d, pool, seq, pos, table, out=out, stream=side)
    side.synchronize()
    pg, row = slots_of(d, seq, pos, table)
    assert torch.equal(out, pool[pg, row])
    # captured once, replayed with other inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.norm_append_kv(d, x, seq, pos, table, pool)
        M.read_kv(d, pool, seq, pos, table, out=out)
    for k in range(3):
        x.copy_(torch.randn((T, d.D), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:, :d.d_c], x[:, :d.d_c])
    assert M.read_device_status() == 0
