"""MI355X-native NVFP4 quantisation engine: fake-quantisation and block-scale selection
(max, MSE over the 126 positive E4M3 scales, Local-Hessian) in HIP kernels for gfx950
behind the C ABI of include/nvfp4.h. ``nvfp4`` is its Python binding; ``kvcache`` is the
key/value cache in NVFP4 with the attention that reads it (include/nvfp4_kv.h); ``rotary``
turns queries and keys by their positions (include/nvfp4_rotary.h)."""
from . import kvcache, nvfp4, rotary  # noqa: F401

__all__ = ["kvcache", "nvfp4", "rotary"]
