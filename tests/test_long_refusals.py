"""More of what the long contexts' calls refuse before they touch the device (CPU only)."""
import test_decode_refusals as step
from test_decode_refusals import INVALID, UNSUPPORTED, batch, lib  # noqa: F401
from test_pages_refusals import keep, move, record


def test_new_lengths_that_overlap_an_input(lib):  # noqa: F811
    """new_len may be ctx_len, budget or seen, not a stretch that begins elsewhere in one of them."""
    at = dict(ctx_len=1 << 20, budget=2 << 20, seen=3 << 20)

    def select(new_len, **kw):
        a = dict(at, **kw)
        return lib.spec_kv_select(record(), batch(B=4, ctx_len=a["ctx_len"]), a["budget"], a["seen"], 0, 0, 4096, 4096, 24, 4096, new_len, None)

    for start in at.values():
        for off in (-12, -4, 4, 12):
            assert select(start + off) == INVALID
        for off in (-16, 16, 0):
            assert select(start + off) != INVALID
    assert select(at["seen"] + 4, seen=None) != INVALID


def test_lists_longer_than_any_context(lib):  # noqa: F811
    """Longer than SPEC_MAX_SLOTS, where an index that goes on by a grid's stride would pass 31 bits."""
    for n in ((1 << 30) + 1, (1 << 31) - 1):
        assert move(lib, most=n) == UNSUPPORTED
        assert move(lib, s=None, most=n) == UNSUPPORTED
        assert keep(lib, m=n) == UNSUPPORTED
        assert keep(lib, s=None, m=n) == UNSUPPORTED
        assert step.keep(lib, m=n) == UNSUPPORTED
