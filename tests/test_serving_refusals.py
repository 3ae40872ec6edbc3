"""Refusals of the serving calls that the binding or the C ABI decides without a device."""
import pytest

from test_serving_abi import ALIGN, OK, P, lib, paged_layout  # noqa: F401 (lib: the fixture)


def test_append_refuses_counts_and_status(lib):  # noqa: F811
    import torch
    import exact_io_aware_100_b200 as fa
    args = [P] * 9
    assert lib.fa_paged_append(*args, paged_layout(tokens=P + 2), 1.0, None) == ALIGN
    assert lib.fa_paged_append(*args, paged_layout(status=P + 1), 1.0, None) == ALIGN
    assert lib.fa_paged_append(*args, paged_layout(tokens=P, status=P, N=0), 1.0, None) == OK
    k = torch.zeros(2, 2, 1, 64, dtype=torch.bfloat16)
    pages, table, lens = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    for name in ("tokens", "status"):
        with pytest.raises(ValueError, match=f"{name}.*int32"):
            fa.paged_append(k, k, pages, pages, table, lens, **{name: torch.zeros(2)})
        with pytest.raises(ValueError, match=f"{name}: expected one per sequence"):
            fa.paged_append(k, k, pages, pages, table, lens, **{name: torch.zeros(3, dtype=torch.int32)})
        with pytest.raises(ValueError, match="CUDA"):
            fa.paged_append(k, k, pages, pages, table, lens, **{name: torch.zeros(2, dtype=torch.int32)})
