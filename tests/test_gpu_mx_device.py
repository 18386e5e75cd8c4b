"""Tensors of a device other than the current one are refused before anything
is launched: a call runs on the current device, where such an address is any
other's or nobody's.  The tensor of another device is a stand-in that has its
type, shape and device and no memory, so the test needs one GPU."""
import pytest
import torch

import mxfp4_routed_expert_k3mx_gb300 as k3mx
from test_gpu_mx_binding import tensors

pytestmark = pytest.mark.gpu


class Elsewhere(torch.Tensor):
    @staticmethod
    def __new__(cls, like):
        return torch.Tensor._make_wrapper_subclass(cls, like.shape, dtype=like.dtype, device="cuda:1")

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(func)


@pytest.mark.parametrize("name", sorted(k3mx._MX_FUNCS))
def test_a_tensor_of_another_device_is_named(cuda_dev, name):
    ok = tensors()[name]
    call = getattr(k3mx, name)
    assert torch.cuda.current_device() == 0
    call(**ok)
    for key, t in ok.items():
        if isinstance(t, torch.Tensor):
            with pytest.raises(TypeError, match=rf"^{key}: .*cuda:0.*cuda:1"):
                call(**dict(ok, **{key: Elsewhere(t)}))
    everything = {k: Elsewhere(t) if isinstance(t, torch.Tensor) else t for k, t in ok.items()}
    with pytest.raises(TypeError, match="cuda:1"):
        call(**everything)
    torch.cuda.synchronize()
    assert k3mx.k3mx_device_status() == (0, 0)
    call(**ok)
