"""Latent pools, the parts that need no device: configurations and null arguments refused
before any device use, the binding's stride and name checks.  CPU only."""
import ctypes

import pytest

import paged_kv_cache_split_gb300 as pkv
from paged_kv_cache_split_gb300 import build as pkv_build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.lib()


@pytest.mark.parametrize("hkv,D,P", [(2, 512, 64), (1, 128, 64), (1, 576, 64), (1, 512, 32), (1, 512, 128)])
def test_unsupported_configurations(lib, hkv, D, P):
    cfg = pkv.make_config(1, hkv, D, "latent", group_size=P)
    h = ctypes.c_void_p()
    assert lib.pkv_pool_create(ctypes.byref(cfg), None, None, ctypes.byref(h)) == pkv.PKV_ERR_INVALID
    assert not h.value


def test_null_pools(lib):
    n = ctypes.c_size_t()
    f = ctypes.c_float
    assert lib.pkv_write_latent(None, 0, 1, None, None, None, 576, None, None, 0, None, f(0), 0, 0, None, 0, 0, None, 0,
                                0, None) == pkv.PKV_ERR_INVALID
    assert lib.pkv_latent_workspace_bytes(None, 1, 1, 1, ctypes.byref(n)) == pkv.PKV_ERR_INVALID
    assert lib.pkv_paged_latent_attention(None, 0, 1, 1, 1, None, 512, None, 64, None, 1, None, 0, f(1), None, None, 0,
                                          None) == pkv.PKV_ERR_INVALID
    assert lib.pkv_latent_prefill_workspace_bytes(None, 1, 1, 1, 1, 0, ctypes.byref(n)) == pkv.PKV_ERR_INVALID
    assert lib.pkv_latent_prefill_attention(None, 0, 1, 1, 1, None, None, None, None, 1, None, 0, f(1), None, None, 0,
                                            None) == pkv.PKV_ERR_INVALID


def test_rope_dim_belongs_to_latent_pools():
    with pytest.raises(ValueError, match="rope_dim"):
        pkv.Pool(1, 1, 128, "bf16", rope_dim=64)


def test_row_stride():
    x = torch.zeros(3, 2, 5, 600)
    assert pkv._row_stride(x[..., :512], "x") == 600
    assert pkv._row_stride(x[:1, :1, :1, :512], "x") == 512
    assert pkv._row_stride(x[:1, :, :1, :512], "x") == 3000
    assert pkv._row_stride(x[:, :1, :1, :512], "x") == 6000
    assert pkv._row_stride(x[0, :, :, 88:], "x") == 600
    assert pkv._row_stride(torch.zeros(0, 2, 5, 64), "x") == 64
    for bad in (x[:, :, :4, :512], x[:, :1, :, :512], x.transpose(0, 1)[..., :512], x[::2][..., :512]):
        with pytest.raises(ValueError, match="evenly spaced"):
            pkv._row_stride(bad, "x")


def test_tensors_that_are_not_on_the_device():
    t = torch.zeros(2, 64, dtype=torch.bfloat16)
    for check in (pkv._dev, pkv._dev_strided):
        with pytest.raises(TypeError, match="CUDA tensor"):
            check(t, torch.bfloat16, "t", (2, 64))
        with pytest.raises(TypeError, match="CUDA tensor"):
            check(None, torch.bfloat16, "t", (2, 64))
