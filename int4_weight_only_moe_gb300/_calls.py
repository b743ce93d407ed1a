"""The compiled form of the Python calls of ``dispatch``, ``lora`` and the router's gradient
(``csrc/calls.cpp``): a call whose tensors are all given and right goes straight to the C
entry. Everything else returns ``None`` there and takes the Python code's steps, which make
what is missing and say what is wrong. So does every call where the extension is not there,
does not load, or was built for another torch or Python, whose tensors it would read wrongly."""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os
import warnings

from ._build import built_for

PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "moe_w4a16_calls.so")

module = None
_refused = None  # the file that did not load


def load():
    """The extension module, once it has been built for this torch and Python; else None."""
    global module, _refused
    if module is None:
        try:
            file = PATH, os.stat(PATH).st_mtime_ns
        except OSError:
            return None
        if file != _refused:
            try:
                module = _load()
            except (ImportError, OSError) as e:
                _refused = file
                warnings.warn(f"the compiled Python calls are not used, the Python steps are taken: {e}")
    return module


def _load():
    import torch  # (whose libraries it links to)
    with open(PATH + ".txt") as f:
        was = f.read()
    if was != built_for(torch.__version__):
        raise ImportError(f"{PATH} was built for {was.strip()}, this is {built_for(torch.__version__).strip()}")
    loader = importlib.machinery.ExtensionFileLoader("moe_w4a16_calls", PATH)
    spec = importlib.util.spec_from_file_location("moe_w4a16_calls", PATH, loader=loader)
    made = importlib.util.module_from_spec(spec)
    loader.exec_module(made)
    return made
