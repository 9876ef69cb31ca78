"""MI355X-native fused late-interaction MaxSim.

score(Q, D) = sum_i max_j <Q_i, D_j>, computed by hand-written gfx950 HIP
kernels behind a C ABI (``include/maxsim.h``), the embedding head that makes
the token rows with the step that trains it (``include/maxsim_encoder.h``), and the
attention layer's operators with a distillation loss (``include/maxsim_layers.h``); the
Python side only marshals arguments.  Submodules:
  binding  -- ctypes binding with the C entry point names (loads libmaxsim.so)
  inputs   -- seeded synthetic inputs (numpy only)
  build    -- compiles libmaxsim.so for gfx950 with hipcc, and _fast.so, the usual small calls past ctypes
"""
__all__ = ["binding", "inputs", "build"]


def __getattr__(name):
    if name in __all__:
        import importlib

        return importlib.import_module("." + name, __name__)
    raise AttributeError(name)
