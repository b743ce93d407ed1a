"""The compiled form of the Python calls of ``dispatch``, ``lora`` and the router's gradient
(``csrc/calls.cpp``): a call whose tensors are all given and right goes straight to the C
entry. Everything else returns ``None`` there and takes the Python code's steps, which make
what is missing and say what is wrong."""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "moe_w4a16_calls.so")

module = None


def load():
    """The extension module, once it has been built."""
    global module
    if module is None and os.path.exists(PATH):
        import torch  # noqa: F401 (whose libraries it links to)
        loader = importlib.machinery.ExtensionFileLoader("moe_w4a16_calls", PATH)
        spec = importlib.util.spec_from_file_location("moe_w4a16_calls", PATH, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
    return module
