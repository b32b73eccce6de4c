"""CPR Gated DeltaNet on B200: a C-ABI CUDA library (libgdn_cpr.so) and its binding.

``rl_train_numerics_b200.gdn`` is the Python binding (imported lazily, since
it loads the CUDA library); ``rl_train_numerics_b200.workloads`` draws the
seeded synthetic inputs.
"""
import importlib

__all__ = ["gdn", "workloads", "build_lib"]


def __getattr__(name):
    if name == "gdn":
        module = importlib.import_module("rl_train_numerics_b200._abi")
    elif name in ("workloads", "build_lib"):
        module = importlib.import_module(f"rl_train_numerics_b200.{name}")
    else:
        raise AttributeError(name)
    globals()[name] = module  # found without this function from now on
    return module
