"""Refusals of the row and shared-prefix calls, before anything is queued (no GPU)."""
import ctypes

import pytest
import torch

import mla_latent_kv_42_b200 as M
from mla_latent_kv_42_b200 import build, synth

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced on the host
MISALIGNED = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return M.load_library()


def swap(args, **at):
    out = list(args)
    for k, v in at.items():
        out[int(k[1:])] = v
    return out


@pytest.mark.parametrize("name", ["mla_norm_append_kv", "mla_norm_append_kv_fp8"])
@pytest.mark.parametrize("d", [synth.PRODUCTION, synth.RUNNING], ids=["production", "running"])
def test_norm_append_refusals(lib, name, d):
    f, cd = getattr(lib, name), M.c_dims(d)
    args = [ctypes.byref(cd), FAKE, d.D, FAKE, FAKE, 1e-6, FAKE, FAKE, FAKE, 2, 4, FAKE, 10, 3, None]
    for at in (1, 6, 7, 8, 11):
        assert f(*swap(args, **{f"_{at}": None})) == -1
    for at in (1, 3, 4, 11):
        assert f(*swap(args, **{f"_{at}": MISALIGNED})) == -4
    assert f(*swap(args, _2=d.D - 8)) == -1 and f(*swap(args, _2=d.D + 4)) == -1
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert f(*swap(args, _5=eps)) == -1
    for at, v in ((9, 0), (10, 0), (12, 0), (13, -1), (13, (1 << 30) + 1)):
        assert f(*swap(args, **{f"_{at}": v})) == -1
    assert f(*swap(args, _13=0)) == 0 and f(*swap(args, _13=0, _1=None)) == 0
    bad = M.c_dims(d)
    bad.d_rope = 6
    assert f(*swap(args, _0=ctypes.byref(bad))) == -2 and f(*swap(args, _0=None)) == -1


@pytest.mark.parametrize("name", ["mla_norm_append_kv", "mla_norm_append_kv_fp8"])
@pytest.mark.parametrize("eps", [1e-50, 1e300])
def test_norm_append_eps_outside_fp32(lib, name, eps):
    """0 or infinity in fp32, where the rows are normalised: a row of zeros would become NaN, any row zeros."""
    d = synth.PRODUCTION
    cd = M.c_dims(d)
    # T, x and pool as in a good call, the misaligned x keeps an accepted eps from being launched
    args = [ctypes.byref(cd), MISALIGNED, d.D, FAKE, FAKE, eps, FAKE, FAKE, FAKE, 2, 4, FAKE, 10, 3, None]
    assert getattr(lib, name)(*args) == -1
    assert getattr(lib, name)(*swap(args, _3=None, _4=None)) == -4  # eps is not used


@pytest.mark.parametrize("name", ["mla_read_kv", "mla_read_kv_fp8"])
def test_read_refusals(lib, name):
    d = synth.PRODUCTION
    f, cd = getattr(lib, name), M.c_dims(d)
    args = [ctypes.byref(cd), FAKE, 10, FAKE, FAKE, FAKE, 2, 4, FAKE, d.D, 3, None]
    for at in (1, 3, 4, 5, 8):
        assert f(*swap(args, **{f"_{at}": None})) == -1
    for at in (1, 8):
        assert f(*swap(args, **{f"_{at}": MISALIGNED})) == -4
    assert f(*swap(args, _9=d.D - 8)) == -1 and f(*swap(args, _9=d.D + 1)) == -1
    for at, v in ((2, 0), (6, 0), (7, 0), (10, -1), (10, (1 << 30) + 1)):
        assert f(*swap(args, **{f"_{at}": v})) == -1
    assert f(*swap(args, _10=0)) == 0


def test_shared_prefix_refusals(lib):
    d = synth.PRODUCTION.with_(n_heads=16)
    f, cd = lib.mla_shared_prefix_attention, M.c_dims(d)
    need = M.workspace_size(d, M.CALL_SHARED_PREFIX_ATTENTION, 2, 256)
    assert need > 0
    args = [ctypes.byref(cd), FAKE, FAKE, 10, FAKE, 4, FAKE, 2, 256, FAKE, 3, FAKE, FAKE, FAKE, need, None]
    for at in (1, 2, 4, 6, 9, 11, 13):
        assert f(*swap(args, **{f"_{at}": None})) == -1
    for at in (1, 2, 11, 12, 13):
        assert f(*swap(args, **{f"_{at}": MISALIGNED})) == -4
    assert f(*swap(args, _14=need - 1)) == -3
    for at, v in ((3, 0), (5, 0), (7, -1), (7, 65536), (8, 0), (8, 257), (10, -1), (10, 5)):
        assert f(*swap(args, **{f"_{at}": v})) == -1
    assert f(*swap(args, _5=1 << 25, _8=(1 << 30) + 1)) == -1
    assert f(*swap(args, _5=1 << 24, _7=200, _8=1 << 30, _14=1 << 62)) == -1  # pages past int32
    assert f(*swap(args, _7=0)) == 0
    assert lib.mla_last_launch_count(M.CALL_SHARED_PREFIX_ATTENTION) == 0


@pytest.mark.parametrize("d", [synth.PRODUCTION, synth.PRODUCTION.with_(n_heads=16), synth.RUNNING,
                               synth.RUNNING.with_(d_c=256, page_size=32)])
def test_shared_prefix_workspace(d):
    ws = lambda B, n: M.workspace_size(d, M.CALL_SHARED_PREFIX_ATTENTION, B, n)
    assert ws(0, 100) == 0 and ws(3, 0) == 0 and ws(3, (1 << 30) + 1) == 0
    for B in (1, 2, 5000):
        for n in (1, 64, 5000):
            assert ws(B, n) >= 8 * B
    for call in range(9, 13):
        assert M.workspace_size(d, call, 5, 100) == 0


def test_binding_refuses_what_the_library_cannot_see():
    d = synth.RUNNING
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):  # host tensors
        M.read_kv(d, torch.zeros((2, 64, d.D), dtype=torch.bfloat16), i32, i32, i32[:, None])


@pytest.mark.gpu
def test_binding_refusals():
    d = synth.RUNNING
    z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")
    i32 = z(3, dtype=torch.int32)
    pool, table, x = z(4, 64, d.D), z(3, 2, dtype=torch.int32), z(3, d.D)
    ok = dict(x=x, seq_idx=i32, pos=i32 + torch.arange(3, device="cuda", dtype=torch.int32), block_table=table,
              pool=pool)
    M.norm_append_kv(d, **ok)
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(x=z(d.D, 3).T), dict(x=z(3, d.D + 4)[:, :d.D]),
                dict(x=z(3, d.D - 8)), dict(x=x[:2]), dict(x=x[0]), dict(x=z(1, d.D).expand(3, -1)),
                dict(pos=i32.long()), dict(pos=i32[:2]), dict(seq_idx=z(6, dtype=torch.int32)[::2]),
                dict(block_table=i32), dict(block_table=table.T), dict(pool=pool[:, :32]), dict(pool=pool.half()),
                dict(pool=pool.flatten(1)), dict(gain_c=z(d.d_c + 8)), dict(gain_c=z(d.d_c).float()),
                dict(gain_r=z(d.d_c))):
        with pytest.raises(ValueError):
            M.norm_append_kv(d, **{**ok, **bad})
    with pytest.raises(M.MLAError):
        M.norm_append_kv(d, **ok, gain_c=z(d.d_c), eps=0.0)
    with pytest.raises(ValueError):
        M.norm_append_kv_fp8(d, **{**ok, "pool": z(4, 64 * d.D, dtype=torch.uint8)})
    for bad in (z(3, d.D).half(), z(2, d.D), z(3, d.D + 4)[:, :d.D]):
        with pytest.raises(ValueError):
            M.read_kv(d, pool, i32, i32, table, out=bad)
    q = z(3, d.n_heads, d.D)
    good = dict(q=q, pool=pool, block_table=table, seq_lens=i32 + 1, max_seq_len=128, shared_pages=i32[:1])
    M.shared_prefix_attention(d, **good)
    for bad in (dict(q=q[:, :3].contiguous()), dict(q=q.half()), dict(block_table=table[:2]),
                dict(seq_lens=i32.long()), dict(shared_pages=table), dict(shared_pages=i32[:1].long()),
                dict(o_lat=z(3, d.n_heads, d.D)), dict(lse=z(3, d.n_heads))):
        with pytest.raises(ValueError):
            M.shared_prefix_attention(d, **{**good, **bad})
    with pytest.raises(M.MLAError):
        M.shared_prefix_attention(d, **{**good, "shared_pages": i32})  # three pages, two in max_seq_len
    with pytest.raises(M.MLAError):
        M.shared_prefix_attention(d, **good, ws=z(16, dtype=torch.uint8))
    assert M.read_device_status() == 0
