"""The workspaces of the calls for prompts follow what a call has to join, not the room in its tables."""
import pytest

from test_serving_library import cache, lib  # noqa: F401


def sizes(lib, positions, page=64, **kw):  # noqa: F811
    return lib.bsg_kv8_attend_window_workspace_size(cache(heads=8, dim=128, page_tokens=page, pages=1 << 20), positions // page,
                                                    kw["B"], kw["T"], 32, 0, 0)


@pytest.mark.parametrize("B,T", [(2, 16384), (40, 300), (64, 64)])
def test_room_for_a_million_positions_takes_no_more(lib, B, T):  # noqa: F811
    """Calls of more blocks of rows than a card has places join nothing, however long their tables
    are: no chunk is made because a table has room for it (two prompts of 16384 behind tables of
    2^20 positions took 8.7 GB)."""
    small = sizes(lib, 32768, B=B, T=T)
    assert sizes(lib, 1 << 20, B=B, T=T) == small <= 256


@pytest.mark.parametrize("B,T", [(1, 17), (1, 300), (3, 1000)])
def test_chunks_are_bounded_by_the_card(lib, B, T):  # noqa: F811
    """Fewer rows than fill the card: at most one chunk of 256 rows for each of some 200 places."""
    for positions in (32768, 1 << 20):
        assert sizes(lib, positions, B=B, T=T) <= (200 * 256 * 4 + 256) * (128 + 2) * 4


def test_every_type_is_sized():
    """A workspace serves any type of the call: the size is the largest over all that there are."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    types = set(re.findall(r"\b(BSG_(?:F32|F16|BF16|F64|F8\w*))\s*=", open(os.path.join(root, "include", "bsgemm.h")).read()))
    text = open(os.path.join(root, "verifiable_quantize_rows_gb300", "csrc", "kv8_more.cu")).read()
    assert len(types) >= 3 and set(re.findall(r"BSG_\w+", re.search(r"kDtypes\[\] = \{([^}]*)\}", text).group(1))) == types
    assert "for (const int dtype : kDtypes)" in text
