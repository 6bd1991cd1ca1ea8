"""Sizes that an int of the library cannot hold are refused by the binding: passed on, they
would be taken for another number (no GPU needed)."""
import pytest
import torch

from attention_forward_gb300 import fa


@pytest.mark.parametrize("pages", [1 << 31, (1 << 32) + 1])
def test_page_tables_wider_than_an_int(pages):
    table = torch.empty((1, pages), dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="fewer than 2\\^31 pages"):
        fa._pages(table, -1, 1)
