"""Arguments that the 4-bit caches' and the axes' helpers refuse (no GPU)."""

import pytest
import torch

import paged_kv_cache_222_gb300 as pkv


@pytest.mark.parametrize("shape", [(), (0,), (36,), (72,), (4, 72), (3, 16, 36), (2, 2, 2, 16, 72)])
@pytest.mark.parametrize("dtype", [torch.uint8, torch.bfloat16])
def test_append_into_what_is_no_cache(shape, dtype):
    c = torch.zeros(shape, dtype=dtype)
    k = torch.zeros((2, 3, 128))
    with pytest.raises(ValueError):
        pkv.append(k, k, torch.zeros(2, dtype=torch.int64), c, c)


@pytest.mark.parametrize("sections", [(1.5, 2), (16, 23.999), (0.5,), (float("nan"), 2)])
def test_parts_of_pairs_are_no_sections(sections):
    with pytest.raises(ValueError):
        pkv.rotary_axes(sections)


def test_whole_numbers_of_any_kind_are():
    import numpy as np
    assert pkv.rotary_axes((2.0, np.int32(1), 3)).tolist() == pkv.rotary_axes((2, 1, 3)).tolist()
    assert pkv.rotary_axes(n for n in (1, 1)).tolist() == [0, 1]
