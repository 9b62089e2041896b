"""More of what the long contexts' calls refuse before they touch the device (CPU only)."""
import pytest
import torch

import speculative_decoding_rejection_verify_gb300 as sv
import test_decode_refusals as step
from speculative_decoding_rejection_verify_gb300 import decode
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


class OnGpu(torch.Tensor):
    """A host tensor that says it is on GPU 0, for checks that come before anything reads it."""

    def get_device(self):
        return 0


def on_gpu(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def gpu_0(monkeypatch, lib):  # noqa: F811
    decode._load()
    monkeypatch.setattr(decode, "_current_device", lambda: 0)
    monkeypatch.setattr(decode, "_raw_stream", lambda index: 0)


def test_scales_that_the_binding_refuses(gpu_0):
    """A scale per page without the other's; a scale per head where entries move, which takes none."""
    k, i, n = on_gpu(2, 16, 2, 64, dtype=torch.float8_e4m3fn), on_gpu(1, 2, dtype=torch.int32), on_gpu(1, dtype=torch.int32)
    x, page, head, lists, w = on_gpu(1, 1, 2, 64, dtype=torch.bfloat16), on_gpu(2, 2), on_gpu(2), on_gpu(1, 2, 3, dtype=torch.int32), on_gpu(2, 2, 16)
    counts = on_gpu(1, 2, dtype=torch.int32)
    calls = dict(append=lambda **s: sv.kv_append(x, x, x, k, k, i, n, **s), attend=lambda **s: sv.paged_attention(x, k, k, i, n, **s),
                 keep=lambda **s: sv.kv_keep(k, k, i, n, i, n, **s), move=lambda **s: sv.kv_move(k, k, i, n, lists, lists, counts, **s))
    for name, call in calls.items():
        for one in (dict(k_scale=page), dict(v_scale=page)):
            with pytest.raises(ValueError, match="both"):
                call(**one)
        with pytest.raises(ValueError, match="_scale: shape"):  # one per page, one per head
            call(k_scale=head, v_scale=page)
        with pytest.raises((ValueError, TypeError), match="v_scale"):
            call(k_scale=page, v_scale=on_gpu(2, 3))
        if name in ("keep", "move"):
            for s in (dict(k_scale=head, v_scale=head), dict(k_scale=head), dict(v_scale=head)):
                with pytest.raises(ValueError, match="per head"):
                    call(**s)
                with pytest.raises(ValueError, match="per head"):
                    call(weight=w, **s)
