"""gmv() of more slots than it takes is refused by the library, and not by an
allocator that is asked for an output of all of them first: nothing larger than
a few elements is allocated on the way to the refusal."""
import pytest
import torch

from moe_grouped_matrix_amd import _binding, _layer, _moe
from test_layer_binding import Ext
from test_layer_checks import gmv_args, lib, swapped  # noqa: F401  (a fixture)
from test_moe_checks import BF16, E, F, F32, I32, UNSUPPORTED, refused, tensor
from test_stream_argument import device, streams  # noqa: F401  (a fixture)


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,k", [(4097, 1), (2 ** 14, 64), (1, 2 ** 20)])
def test_nothing_is_allocated(streams, monkeypatch, T, k, weighted):  # noqa: F811
    made = []
    for module in (_moe, _layer):
        monkeypatch.setattr(module, "_empty", lambda shape, dtype, dev, stream: (made.append(torch.Size(shape)), device(1, dtype=dtype))[1])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x77, raising=False)
    monkeypatch.setattr(_moe, "_ext", Ext())
    monkeypatch.setattr(_layer, "_current", lambda t: 0)
    _layer._gmv_workspace.cache_clear()

    class Library:
        def gmm_gmv_workspace(self, slots, N, weighted, need):
            return _binding.GMM_E_UNSUPPORTED

        def gmm_gmv_run(self, *args):
            return _binding.GMM_E_UNSUPPORTED

        def gmm_last_error(self, h):
            return b"more than 4096 slots"

    monkeypatch.setattr(_binding, "_lib", Library())
    x, q = device(T, 32), device(2, 4096, 16, dtype=torch.uint8)
    s, ids = device(2, 1, 1, 4096, dtype=torch.float32), device(T, k, dtype=torch.int32)
    w = device(T, k, dtype=torch.float32) if weighted else None
    with pytest.raises(_binding.GmmUnsupported, match="4096 slots"):
        _layer.gmv(x, q, ids, rhs_format="int4", rhs_scale=s, weights=w)
    assert [n.numel() for n in made] == [0]
    _layer._gmv_workspace.cache_clear()


def test_the_library_refuses_by_the_slots(lib):  # noqa: F811
    """(whatever the output holds)"""
    ok = gmv_args(T=4097, k=1)
    refused(lib, UNSUPPORTED, "4096 slots", "gmv", *swapped(ok, a6=tensor(None, F32, 0, 1, 24)))
    refused(lib, UNSUPPORTED, "4096 slots", "gmv", *swapped(ok, a4=tensor(E, I32, 2049, 2), a6=tensor(None, BF16, 0, 24)))
    refused(lib, UNSUPPORTED, "64 choices", "gmv", *swapped(ok, a4=tensor(E, I32, 1, 1 << 20), a6=tensor(F, F32, 0, 24)))
