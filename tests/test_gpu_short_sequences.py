"""Sequences that are shorter than the prefix the rest of the batch shares, down to one token and up to one
short of it: they attend to their own pages alone, in pieces of their own. Bounds as in
test_gpu_shared_prefix."""
import numpy as np
import pytest
import torch

import mla_latent_kv_42_b200 as M
from mla_latent_kv_42_b200 import build, synth
from test_gpu_shared_prefix import Case, batch

pytestmark = pytest.mark.gpu

P, R = synth.PRODUCTION, synth.RUNNING


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    M.load_library()
    M.read_device_status()


@pytest.mark.parametrize("d,B,shared", [
    (R, 16, 40), (R, 2, 100), (R.with_(n_heads=3), 45, 33), (R.with_(n_heads=7, dtype="fp16"), 30, 64),
    (R.with_(n_heads=1), 150, 20), (R.with_(n_heads=16, page_size=16), 13, 90), (R.with_(n_heads=5, page_size=48), 64, 40),
    (R.with_(n_heads=9, d_c=16, d_rope=16, page_size=32), 300, 30), (P.with_(n_heads=16), 20, 40), (P.with_(n_heads=48), 30, 9),
])
@pytest.mark.parametrize("every", [1, 2, 7])
def test_shorter_than_the_prefix(d, B, shared, every):
    """One sequence in ``every``; every partial that is read was written by this call (the workspace
    holds NaN before), and the call repeats itself bit for bit."""
    n = shared * d.page_size
    lens = batch(B, n, [1, 70, 0, 200])
    short = np.asarray([n - 1, 1, n // 2 + 3, n - 63, 64, 65, n - d.page_size])
    lens[::every] = short[np.arange(len(lens[::every])) % len(short)].clip(1)
    c = Case(d, lens, shared, seed=B, spare=5)
    top = c.longest if every > 1 else n + 60
    ws = torch.empty(M.workspace_size(d, M.CALL_SHARED_PREFIX_ATTENTION, B, top), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    o, lse = c.run(ws=ws, longest=top)
    assert M.read_device_status() == 0
    c.check(o, lse)
    ws.fill_(0xFF)
    o2, lse2 = c.run(ws=ws, longest=top)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("heads", [3, 8])
def test_short_rejected_and_not_a_number(heads):
    """A short sequence with a bad page is rejected alone, one with a NaN row keeps it to itself."""
    d = R.with_(n_heads=heads)
    n = 30 * d.page_size
    lens = batch(20, n, [5, 90])
    lens[[2, 3, 9, 17]] = [n - 1, n - 5, n - 1, 700]
    c = Case(d, lens, 30, seed=4)
    o, lse = c.run()
    c.check(o, lse)
    c.table[3, 20] = -1
    c.pool[c.table[9, 12].long(), 7] = float("nan")
    got, got_l = c.run()
    assert M.read_device_status() == -7
    same = [b for b in range(20) if b not in (3, 9)]
    assert torch.equal(got[same], o[same]) and torch.equal(got_l[same], lse[same])
    assert not bool(got[3].any()) and bool((got_l[3] == -float("inf")).all())
    assert bool(got[9].isnan().all()) and bool(got_l[9].isnan().all())


@pytest.mark.parametrize("d,B,shared", [(P.with_(n_heads=16), 20, 40), (P, 5, 3), (P.with_(n_heads=1), 300, 2), (R, 16, 40),
                                        (R.with_(d_c=256, page_size=32), 4, 3)],
                         ids=["packed", "h128", "plan-kernel", "narrow", "generic"])
def test_a_batch_of_rejected_sequences_only(d, B, shared):
    """Every length is zero: outputs of zeros, lse of -inf, the error recorded, nothing left in the way."""
    c = Case(d, batch(B, shared * d.page_size, [1, 70]), shared, seed=9)
    good, good_l = c.run()
    assert M.read_device_status() == 0
    kept = c.lens.clone()
    c.lens.zero_()
    o, lse = c.run()
    assert M.read_device_status() == -8
    assert not bool(o.any()) and bool((lse == -float("inf")).all())
    c.lens.copy_(kept)
    o, lse = c.run()
    assert M.read_device_status() == 0 and torch.equal(o, good) and torch.equal(lse, good_l)
