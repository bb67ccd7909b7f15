"""GB300-native FP32 SGEMM: C = alpha*A*B + beta*C, row-major, behind a C ABI; and around it the
linear layer of a language model (low-rank adapters, 8-bit activation checkpoints).

The compute path is ``libsgemm`` (hand-written CUDA for sm_103a, built from
``csrc/``); ``binding`` marshals torch tensors to it and nothing else.  The
binding is imported lazily so that the seeded input generators in
``workloads`` can be used without the CUDA library; calling any SGEMM entry
point without a built library raises immediately (there is no CPU fallback).
"""

_LAYERS = ("lora_into", "lora_backward_into", "act8_empty", "act8_store_into", "act8_load_into",
           "act8_grad_into", "act8_weight_grad_into")
__all__ = ["sgemm", "sgemm_host", "sgemm_into", *_LAYERS, "library_path", "workloads"]


def __getattr__(name):
    if name in ("sgemm", "sgemm_host", "sgemm_into", "library_path", "lib", *_LAYERS):
        from . import binding
        return getattr(binding, name)
    raise AttributeError(name)
