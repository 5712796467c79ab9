"""Tensors that have sizes, strides, a dtype and a device, but no memory: for refusals that
the binding makes before it looks at a GPU.  (Their address is null, which the library
refuses too, so a call that is not refused ends before a launch.)"""
import torch


class Standin(torch.Tensor):
    @staticmethod
    def __new__(cls, size, strides=None, dtype=torch.float32, device="cuda:0"):
        return torch.Tensor._make_wrapper_subclass(cls, size, strides=strides, dtype=dtype,
                                                   device=torch.device(device))

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise RuntimeError("%s of a tensor without memory" % func)
