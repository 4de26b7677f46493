"""dense_attn at widths, caps and masks where its kernels' limits lie; tolerances as in test_dense_attn.py."""

import pytest
import torch

import lightning_indexer_top_gb300 as L
from test_dense_attn import DTYPES, Case

# dk, dv of K and V apart / of a latent; every one with two to eight key splits that a cluster merges.  Narrow keys
# beside wide values, and latents just past a step of the value width: the merged rows are longer than Q, K, V and the
# scores, or nearly so.
NARROW = [(1, 128), (4, 128), (8, 128), (12, 126), (13, 128), (4, 65)]
NARROW_LATENT = [(1, 1), (8, 8), (16, 16), (20, 20), (12, 5), (129, 129), (136, 136), (140, 140), (144, 130), (144, 144)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv", NARROW)
def test_merged_rows_of_narrow_keys(dtype, dk, dv):
    for T, n_kv in ((5, [256, 90]), (1, [200]), (9, [64, 40, 60])):
        c = Case(n_kv, T, 8, 1, dk, dv=dv, dtype=dtype, page=16, seed=41)
        c.check(*c.run(), what=(T, n_kv))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv", NARROW_LATENT)
def test_merged_rows_of_narrow_latents(dtype, dk, dv):
    for T, Hq, n_kv in ((1, 16, [256, 90]), (5, 8, [200, 33]), (3, 5, [64])):
        c = Case(n_kv, T, Hq, 1, dk, dv=dv, dtype=dtype, latent=True, seed=42)
        c.check(*c.run(), what=(T, Hq, n_kv))
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv,latent", [(576, 128, False), (576, 64, False), (529, 128, False), (528, 128, False),
                                          (549, 64, False), (576, 128, True), (573, 40, True), (576, 512, False)])
def test_wide_keys_of_many_rows(dtype, dk, dv, latent):
    # 64 rows of keys this wide are more than a CTA's shared memory holds
    for T, Hq in ((5, 8), (17, 1)):
        c = Case([150, 33], T, Hq, 1, dk, dv=dv, dtype=dtype, page=16, latent=latent, seed=43)
        c.check(*c.run(), what=(T, Hq))
