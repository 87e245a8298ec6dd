"""The binding's checks of a decode's tensors, which come before any launch (CPU
tensors: nothing is launched here)."""
from __future__ import annotations

import pytest
import torch

from paged_mla_decode_02_gb300 import mla


def tensors(**other):
    t = dict(q_nope=torch.zeros((2, 16, 512), dtype=torch.bfloat16), q_pe=torch.zeros((2, 16, 64), dtype=torch.bfloat16),
             ckv_cache=torch.zeros((3, 16, 512), dtype=torch.bfloat16),
             kpe_cache=torch.zeros((3, 16, 64), dtype=torch.bfloat16),
             out=torch.zeros((2, 16, 512), dtype=torch.bfloat16), lse=torch.zeros((2, 16)))
    t.update({k: t[k].to(v) for k, v in other.items()})
    return t


def test_matching_tensors_pass():
    mla._check_layouts(**tensors(), page_size=16)
    mla._check_layouts(**tensors(out=torch.float32), page_size=16)


# fewer bytes than the kernels write or read there
@pytest.mark.parametrize("other", [dict(lse=torch.bfloat16), dict(lse=torch.float16), dict(lse=torch.uint8),
                                   dict(q_pe=torch.uint8), dict(q_pe=torch.float8_e4m3fn), dict(q_pe=torch.float32)])
def test_other_types_are_refused(other):
    with pytest.raises(ValueError):
        mla._check_layouts(**tensors(**other), page_size=16)
