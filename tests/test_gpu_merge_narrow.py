"""Decode at latent widths below 128 with more splits than lanes hold columns: the merge of the
split-KV partials shuffles its weights across the whole warp, also from lanes without columns."""
import numpy as np
import pytest
import torch

import mla_latent_kv_42_b200 as M
import oracle as O
from mla_latent_kv_42_b200 import build, synth
from parity import CacheCase, assert_parity, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    M.load_library()
    M.read_device_status()


@pytest.mark.parametrize("d_c,d_rope,heads", [(16, 16, 8), (48, 16, 3), (112, 32, 16), (136, 24, 9)])
def test_split_decode_at_narrow_latents(d_c, d_rope, heads):
    import dataclasses
    w = dataclasses.replace(synth.workload("running_b16_n4096_l12_bf16"),
                            dims=synth.RUNNING.with_(d_c=d_c, d_rope=d_rope, n_heads=heads))
    d = w.dims
    lens = np.array([2000, 700])
    case = CacheCase(w, cached=lens, paging="shuffled", spare_tokens=0)
    q = synth.synthetic_query(w, len(lens), scale=3.0)
    assert M.workspace_size(d, M.CALL_DECODE_ATTENTION, 2, 2000) > 0  # it splits
    o, lse = M.decode_attention(d, q.cuda(), case.pool, case.block_table,
                                torch.from_numpy(lens.astype(np.int32)).cuda(), 2000)
    assert M.read_device_status() == 0
    for b in range(2):
        ref_o, ref_l = O.latent_attention(O.as64(q[b]), O.as64(case.prefix(b)), d)
        assert_parity(to64(o[b]), ref_o, f"sequence {b}")
        np.testing.assert_allclose(to64(lse[b]), ref_l, rtol=0, atol=2e-2)
