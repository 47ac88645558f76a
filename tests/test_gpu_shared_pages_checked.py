"""A bad id in ``shared_pages`` alone (the block table is whole) rejects every sequence that has the prefix,
whether the call packs the rows of the batch or not, and no other."""
import pytest

import mla_latent_kv_42_b200 as M
from mla_latent_kv_42_b200 import build, synth
from test_gpu_shared_prefix import GENERIC, Case, batch

pytestmark = pytest.mark.gpu

P, R = synth.PRODUCTION, synth.RUNNING


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    M.load_library()
    M.read_device_status()


@pytest.mark.parametrize("d,B,shared", [
    (P.with_(n_heads=16), 12, 40), (P.with_(n_heads=16), 4, 3), (P.with_(n_heads=16), 300, 2), (P, 6, 3), (P, 1, 4),
    (P.with_(n_heads=1), 5000, 1), (R, 12, 5), (R, 1, 5), (GENERIC, 6, 3), (P.with_(page_size=32), 5, 3),
], ids=["packed", "few", "many", "h128", "one", "plan-kernel", "narrow", "narrow-one", "generic", "pages-of-32"])
@pytest.mark.parametrize("bad", ["past", "negative"])
def test_bad_shared_page(d, B, shared, bad):
    lens = batch(B, shared * d.page_size, [1, 70, 0, 130])
    idle = [2] if B > 2 else []
    lens[idle] = 3
    c = Case(d, lens, shared, seed=21)
    exact = d is not GENERIC and d.page_size == 64
    o, lse = c.run()
    assert M.read_device_status() == 0
    some = range(B) if B <= 12 else [0, 1, 2, 3, B - 1]
    c.check(o, lse, skip=set(range(B)) - set(some), exact_lse=exact)
    c.shared[shared - 1] = len(c.pool) if bad == "past" else -1
    o, lse = c.run()
    assert M.read_device_status() == -7
    has = [b for b in range(B) if b not in idle]
    assert not bool(o[has].any()) and bool((lse[has] == -float("inf")).all())
    c.check(o, lse, skip=has, exact_lse=exact)
