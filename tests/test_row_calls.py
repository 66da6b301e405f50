"""Calls of the operators over vocabulary rows as the host sees them: what the package needs of torch when it is
imported, workspaces, and refusals (the pointers here are never followed)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import causal_draft_correction_amd as dca
from causal_draft_correction_amd.rows import Beam, Logits, _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3


def test_the_package_imports_without_the_private_stream_name():
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
            "    del torch._C._cuda_getCurrentRawStream\n"
            "import causal_draft_correction_amd as dca\n"
            "from causal_draft_correction_amd import rows\n"
            "class One:\n"
            "    cuda_stream = 7\n"
            "torch.cuda.current_stream = lambda gpu: One\n"
            "assert rows._stream(0) == 7 and dca.top_logits is rows.top_logits\n")
    got = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert got.returncode == 0, got.stderr
