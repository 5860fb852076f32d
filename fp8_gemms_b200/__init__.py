"""FP8 training GEMMs with dynamic tensorwise scaling for B200 (sm_100a).

The compute path is libfp8lm.so (C ABI in include/lm_fp8.h); ``_lib`` is its
ctypes binding and ``api`` adds PyTorch-allocated buffers around it.  Both
import the library eagerly and fail if it is not built; the row operators and rotary
positions also need ``_native`` (a C++ module), and fail when they are called without it.  ``synthetic`` holds
the seeded input generators and needs no GPU.
"""
__all__ = ["api", "synthetic"]
