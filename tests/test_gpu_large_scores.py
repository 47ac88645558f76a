"""Attention scores of thousands: the softmax reference has to follow them closely enough for weights of
the element type (fp16 holds 2^-14 to 2^16), in every call of the tensor-core kernel.

Rows and queries are chosen so that every score is exact in fp32: a row is A b_d (A = 3.5, b_d = +-1)
but for its noise columns, multiples of A / 2, a query k b_d with |k| <= 250 but for small integers; all
products are multiples of 1/4 with sums below 2^24 of them. (A is 448 / 2^7, so that an e4m3 row with its
power-of-two scale holds the same values.) What is left, for natural scores of at most S: the factor
log2(e) / sqrt(d_h + d_h^R) is rounded to fp32, and so is each exponent and the reference, 2^-24 of the
score each; 8 such units, 2^-21 S =: e, cover a weight's logarithm and the lse. exp2 and the sums
add less than 2^-17. Half a step u of the element type each for the weights and for o, and where the
weights are fp16 half its smallest subnormal, 2^-25, per token (the largest weight is 1 or more).
"""
import pytest
import torch

import mla_latent_kv_42_b200 as M
from mla_latent_kv_42_b200 import build, synth

pytestmark = pytest.mark.gpu

A, BASE = 3.5, 436  # columns from BASE on: 76 of noise, then the rotated part of the base again
P = synth.PRODUCTION


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    M.load_library()
    M.read_device_status()


def i32(a):
    return torch.as_tensor(a, dtype=torch.int32, device="cuda")


def make(d, n, k, seed):
    """(rows [n, D], base [D]); the score against k * base steps up twice along the rows (k > 0; down for
    k < 0) by far more than a rescaling threshold."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    b = torch.randint(0, 2, (d.D,), device="cuda", generator=g).double() * 2 - 1
    rows = (A * b).repeat(n, 1)
    third = torch.arange(n, device="cuda") * 3 // max(n, 1)
    rows[third < 1, 3] *= -1
    rows[third < 2, 5] *= -1
    rows[:, BASE:512] = torch.randint(-2, 3, (n, 512 - BASE), device="cuda", generator=g).double() * (A / 2)
    return rows, b


def queries(d, B, b, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = (k * b).repeat(B, d.n_heads, 1)
    q[..., BASE:512] = torch.randint(-2, 3, (B, d.n_heads, 512 - BASE), device="cuda", generator=g).double()
    return q


def check(d, q, rows_of, o, lse, exact_lse, weights):
    u = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[d.dtype]
    uw = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[weights]
    scale = (d.d_head + d.d_rope) ** -0.5
    for b in range(len(q)):
        rows = rows_of(b)
        s = q[b] @ rows.T * scale
        ref_l = s.logsumexp(1)
        p = (s - ref_l[:, None]).exp()
        v = rows[:, :d.d_c]
        ref, mag = p @ v, p @ v.abs()
        err = 2.0 ** -21 * s.abs().amax(1) + 2.0 ** -17
        tol = uw * mag + u * ref.abs() + 2 * err[:, None] * mag + 2.0 ** -24
        if weights == "fp16":
            tol = tol + len(rows) * 2.0 ** -25 * A
        off = (o[b].double() - ref).abs()
        assert bool((off <= tol).all()), (b, len(rows), float((off / tol).nan_to_num(1e9).max()))
        assert bool(((lse[b].double() - ref_l).abs() <= err + (0 if exact_lse else uw)).all()), (b, len(rows))


@pytest.mark.parametrize("k", [24, -24, 250, -250])
@pytest.mark.parametrize("heads,dtype", [(16, "fp16"), (16, "bf16"), (64, "fp16"), (128, "fp16"), (128, "bf16")])
def test_shared_prefix(heads, dtype, k):
    d = P.with_(n_heads=heads, dtype=dtype)
    page, shared, own = d.page_size, 30, [1, 70, 129, 300, 64, 650]
    B = 24
    rows, b = make(d, (shared + 11 * len(own)) * page, k, heads)
    rows = rows[torch.randperm(len(rows), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))] \
        if heads == 64 else rows
    pool = rows.to(synth.storage_dtype(d)).view(-1, page, d.D)
    assert torch.equal(pool.double().view(-1, d.D), rows)
    lens = [shared * page + own[i % len(own)] for i in range(B)]
    table = [list(range(shared)) + [shared + 11 * (i % len(own)) + j for j in range(11)] for i in range(B)]
    q = queries(d, B, b, k, heads)
    o, lse = M.shared_prefix_attention(d, q.to(pool.dtype), pool, i32(table), i32(lens), max(lens),
                                       i32(list(range(shared))))
    assert M.read_device_status() == 0
    check(d, q, lambda i: rows.view(-1, page, d.D)[table[i]].view(-1, d.D)[:lens[i]], o, lse, True, dtype)


@pytest.mark.parametrize("k", [24, -24, 250, -250])
@pytest.mark.parametrize("dtype,fp8", [("fp16", False), ("bf16", False), ("bf16", True), ("fp16", True)])
def test_decode(dtype, fp8, k):
    d = P.with_(dtype=dtype)
    # ten sequences of each length over the same pages: several tiles and items to each pair of SMs
    page, lens = d.page_size, [3000, 1, 64, 700, 5000, 129]
    used = [-(-n // page) for n in lens]
    rows, b = make(d, sum(used) * page, k, 7)
    table = [[sum(used[:i]) + min(j, n - 1) for j in range(max(used))] for i, n in enumerate(used)] * 10
    lens = lens * 10
    q = queries(d, len(lens), b, k, 7)
    e = synth.storage_dtype(d)
    if fp8:
        pool = torch.zeros((sum(used), M.fp8_page_bytes(d)), dtype=torch.uint8, device="cuda")
        n = page * d.D
        pool[:, :n] = (rows * 128).to(torch.float8_e4m3fn).view(torch.uint8).view(len(pool), n)
        pool[:, n:] = torch.full((len(pool), 2 * page), 2.0 ** -7, device="cuda").view(torch.uint8)
        assert torch.equal(M.read_kv_fp8(d, pool, i32([0] * 128), i32(list(range(128))), i32([[0, 1]])).double(),
                           rows[:128])
        o, lse = M.decode_attention_fp8(d, q.to(e), pool, i32(table), i32(lens), max(lens))
    else:
        pool = rows.to(e).view(-1, page, d.D)
        o, lse = M.decode_attention(d, q.to(e), pool, i32(table), i32(lens), max(lens))
    assert M.read_device_status() == 0
    check(d, q, lambda i: rows.view(-1, page, d.D)[table[i]].reshape(-1, d.D)[:lens[i]], o, lse, False,
          "fp16" if fp8 else dtype)


@pytest.mark.parametrize("k", [24, -250])
@pytest.mark.parametrize("d", [synth.RUNNING.with_(dtype="fp16"), synth.RUNNING], ids=["fp16", "bf16"])
def test_narrow_rows(d, k):
    """The warp-MMA kernel, by the same construction: noise in the last latent columns."""
    page, shared, B = d.page_size, 20, 9
    g = torch.Generator(device="cuda").manual_seed(3)
    b = torch.randint(0, 2, (d.D,), device="cuda", generator=g).double() * 2 - 1
    rows = (A * b).repeat((shared + 2 * B) * page, 1)
    rows[:, 100:128] = torch.randint(-2, 3, (len(rows), 28), device="cuda", generator=g).double() * (A / 2)
    rows[:len(rows) // 3, 3] *= -1
    q = (k * b).repeat(B, d.n_heads, 1)
    q[..., 100:128] = torch.randint(-2, 3, (B, d.n_heads, 28), device="cuda", generator=g).double()
    lens = [shared * page + 1 + 13 * i for i in range(B)]
    table = [list(range(shared)) + [shared + 2 * i, shared + 2 * i + 1] for i in range(B)]
    pool = rows.to(synth.storage_dtype(d)).view(-1, page, d.D)
    o, lse = M.shared_prefix_attention(d, q.to(pool.dtype), pool, i32(table), i32(lens), max(lens),
                                       i32(list(range(shared))))
    assert M.read_device_status() == 0
    check(d, q, lambda i: rows.view(-1, page, d.D)[table[i]].view(-1, d.D)[:lens[i]], o, lse, True, d.dtype)
