"""A bounded wait of prompt attention that runs out, without faulting the GPU: in a copy of the
library with a 1 ms limit the first CTA does not start one copy of a K or V tile, so that the
waits for it cannot end. The call comes back with a wait's bit in the device error word, every
role of the kernel has ended, and the next call with the hook off is correct."""
import ctypes

import pytest
import torch

import paged_kv_cache_154_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def test_lib():
    from paged_kv_cache_154_gb300 import build
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    L = ctypes.CDLL(build.build_variant("pa_waittest", ["-DPA_TEST_HOOKS",
                                                        "-DPA_WAIT_LIMIT_NS=1000000ull"]))
    for name, (args, res) in pa._SIGS.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    L.pa_test_skip_tile.argtypes = [ctypes.c_int]
    L.pa_test_skip_tile.restype = ctypes.c_int
    return L


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tile", [0, 1, 6, 9])      # K or V, of the first or a later task's tiles
def test_a_tile_that_never_comes(test_lib, monkeypatch, d, tile):
    T, H, G = 1500, 8, 4
    x = torch.randn((T, H + 2 * G, d), generator=torch.Generator().manual_seed(d)).to(
        torch.bfloat16).cuda()
    start = torch.tensor([0, 700, T], dtype=torch.int32, device="cuda")

    def call(out):
        pa.prompt_attention(out, x[:, :H], x[:, H:H + G], x[:, H + G:], start, 800, d ** -0.5)
        torch.cuda.synchronize()

    want, got = (torch.zeros((T, H, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    call(want)
    assert pa.device_error() == 0
    monkeypatch.setattr(pa, "_lib", test_lib)
    assert test_lib.pa_test_skip_tile(tile) == 0
    call(got)
    code = pa.device_error()
    assert code & (pa.DEVERR_WAIT_FULL | pa.DEVERR_WAIT_EMPTY), hex(code)
    assert not code & (pa.DEVERR_BAD_BLOCK | pa.DEVERR_BAD_SLOT | pa.DEVERR_WORKSPACE), hex(code)
    assert test_lib.pa_test_skip_tile(-1) == 0
    got.zero_()
    call(got)
    assert (code := pa.device_error()) == 0, hex(code)
    assert torch.equal(got, want)
