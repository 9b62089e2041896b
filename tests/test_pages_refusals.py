"""What the operators of page scales and eviction refuse before they touch the device (CPU only)."""
import ctypes

import pytest
import torch

import speculative_decoding_rejection_verify_gb300 as sv
from speculative_decoding_rejection_verify_gb300 import decode
from test_decode_refusals import (BAD_BATCHES, BAD_CACHES, INVALID, OK, UNSUPPORTED, WORKSPACE, batch, cache, heads,  # noqa: F401
                                  lib)

E4M3 = decode.DTYPE_E4M3


def f8(**kw):
    return cache(**dict(dict(dtype=E4M3), **kw))


def scales(**kw):
    return ctypes.byref(decode.PageScalesStruct(*dict(dict(k=4096, v=4096, layer_stride=32), **kw).values()))


def record(**kw):
    a = dict(weight=4096, position=4096, layer_stride=0, layers=1, num_pages=4, page_size=16, heads=8)
    a.update(kw)
    return ctypes.byref(decode.RecordStruct(*a.values()))


def append(lib, c=None, s=True, b=None):
    return lib.spec_kv_append_ex(heads(), heads(), heads(), heads(), 8, c or f8(), scales() if s is True else s, b or batch(), None, None, None)


def attend(lib, c=None, s=True, b=None, lse=4096, ws=4096):
    return lib.spec_paged_attention_ex(heads(), heads(), 8, c or f8(), scales() if s is True else s, b or batch(), None, 0.1, lse, ws, 1 << 30, None)


def keep(lib, c=None, s=True, r=True, b=None, path=4096, n=4096, m=3):
    return lib.spec_kv_keep_ex(c or f8(), scales() if s is True else s, record() if r is True else r, b or batch(), path, n, m, None)


def weigh(lib, c=None, s=True, r=True, b=None, q=True, n=8, scale=0.1, lse=4096):
    return lib.spec_kv_weigh(heads() if q is True else q, n, c or f8(), scales() if s is True else s, b or batch(), None, scale, lse,
                             record() if r is True else r, None, None)


def select(lib, r=True, b=None, budget=4096, first=0, recent=0, src=4096, dst=4096, most=24, moves=4096, out=4096):
    return lib.spec_kv_select(record() if r is True else r, b or batch(), budget, None, first, recent, src, dst, most, moves, out, None)


def move(lib, c=None, s=True, r=True, b=None, src=4096, dst=4096, moves=4096, most=24):
    return lib.spec_kv_move(c or f8(), scales() if s is True else s, record() if r is True else r, b or batch(), src, dst, moves, most, None)


CALLS = [append, attend, keep, weigh, move]


@pytest.mark.parametrize("call", CALLS)
def test_bad_caches_batches_and_scales(lib, call):  # noqa: F811
    for change, status in BAD_CACHES:
        name = next(iter(change))
        if "scale" in name or (call is weigh and name == "v"):
            continue
        assert call(lib, c=cache(**dict(dict(dtype=E4M3), **change))) == status, change
    for change, status in BAD_BATCHES:
        if "T" in change and call in (keep, move):
            continue
        assert call(lib, b=batch(**change)) == status, change
    for bad in (scales(k=None), scales(k=4098), scales(layer_stride=-1)):
        assert call(lib, s=bad) == INVALID
    if call is not weigh:  # which uses no values
        for bad in (scales(v=None), scales(v=4097)):
            assert call(lib, s=bad) == INVALID
    assert call(lib, c=cache()) == INVALID                    # page scales of a bf16 cache
    assert call(lib, c=f8(k_scale=4096)) == INVALID           # two kinds of scale
    if call is not weigh:
        assert call(lib, c=f8(v_scale=4096)) == INVALID
    assert call(lib, b=batch(B=0)) == OK


@pytest.mark.parametrize("call", [keep, weigh, move])
def test_records(lib, call):  # noqa: F811
    for bad in (dict(weight=4098), dict(position=4097), dict(layer_stride=-1), dict(layers=0), dict(num_pages=0), dict(heads=0),
                dict(layers=2), dict(num_pages=5), dict(page_size=32), dict(heads=4)):
        assert call(lib, r=record(**bad)) == INVALID, bad
    assert call(lib, r=record(page_size=24)) == UNSUPPORTED


def test_keep_arguments(lib):  # noqa: F811
    assert keep(lib, m=-1) == INVALID
    assert keep(lib, m=65) == UNSUPPORTED
    assert keep(lib, path=None) == INVALID
    assert keep(lib, n=None) == INVALID
    assert keep(lib, m=0, path=None, n=None) == OK
    assert keep(lib, b=batch(B=65536)) == UNSUPPORTED


def test_weigh_arguments(lib):  # noqa: F811
    assert lib.spec_kv_weigh(heads(), 8, None, None, batch(), None, 0.1, 4096, record(), None, None) == INVALID
    assert weigh(lib, r=None) == INVALID
    assert weigh(lib, r=record(weight=None)) == INVALID
    assert weigh(lib, q=None) == INVALID
    assert weigh(lib, lse=None) == INVALID
    assert weigh(lib, n=0) == INVALID
    assert weigh(lib, n=12) == INVALID
    assert weigh(lib, n=8 * 129) == UNSUPPORTED
    assert weigh(lib, scale=float("nan")) == INVALID
    assert weigh(lib, b=batch(T=65)) == UNSUPPORTED
    assert weigh(lib, b=batch(T=0)) == OK
    assert weigh(lib, c=f8(v=None), b=batch(T=0)) == OK  # values are not used


def test_select_arguments(lib):  # noqa: F811
    assert select(lib, r=None) == INVALID
    for bad in (dict(weight=None), dict(weight=4097), dict(position=4098), dict(layers=0), dict(num_pages=-1), dict(heads=0), dict(page_size=0),
                dict(layer_stride=-4), dict(weight=4100), dict(position=4104), dict(layer_stride=6)):
        assert select(lib, r=record(**bad)) == INVALID, bad
    assert select(lib, r=record(page_size=4)) == UNSUPPORTED
    assert select(lib, r=record(heads=65536)) == UNSUPPORTED
    for change, status in BAD_BATCHES:
        if "T" not in change:
            assert select(lib, b=batch(**change)) == status
    assert select(lib, first=-1) == INVALID
    assert select(lib, recent=-1) == INVALID
    assert select(lib, r=record(position=None), first=1) == INVALID
    assert select(lib, r=record(position=None), recent=1) == INVALID
    assert select(lib, most=23) == INVALID  # half of 3 pages of 16
    assert select(lib, most=-1) == INVALID
    for missing in ("budget", "src", "dst", "moves", "out"):
        assert select(lib, **{missing: None}) == INVALID
    assert select(lib, b=batch(B=65536)) == UNSUPPORTED
    assert select(lib, b=batch(B=0)) == OK


def test_move_arguments(lib):  # noqa: F811
    assert move(lib, most=-1) == INVALID
    for missing in ("src", "dst", "moves"):
        assert move(lib, **{missing: None}) == INVALID
    assert move(lib, most=0, src=None, dst=None, moves=None) == OK
    assert move(lib, b=batch(B=65536)) == UNSUPPORTED


def test_attention_arguments(lib):  # noqa: F811
    assert attend(lib, ws=None) == WORKSPACE
    assert attend(lib, b=batch(T=65)) == UNSUPPORTED
    assert attend(lib, lse=4098) == INVALID
    assert attend(lib, b=batch(T=0)) == OK


def test_structs_match_the_header(tmp_path):
    import shutil
    import subprocess
    from test_abi import INCLUDE
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    pairs = (("spec_kv_page_scales_t", decode.PageScalesStruct, decode._pack_scales), ("spec_kv_record_t", decode.RecordStruct, decode._pack_record))
    body = "".join(f'printf("%zu\\n", sizeof({n}));' + "".join(f'printf("%zu\\n", offsetof({n}, {f[0]}));' for f in s._fields_) for n, s, _ in pairs)
    src = tmp_path / "s.c"
    src.write_text('#include "spec_decode.h"\n#include <stdio.h>\nint main(void) {' + body + "return 0;}\n")
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", INCLUDE, str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [n for _, s, _ in pairs for n in [ctypes.sizeof(s)] + [getattr(s, f[0]).offset for f in s._fields_]]
    for _, cls, pack in pairs:
        values = list(range(1, len(cls._fields_) + 1))
        s = cls.from_buffer_copy(pack(*values))
        assert [getattr(s, f[0]) for f in cls._fields_] == values


def test_the_binding_refuses(lib):  # noqa: F811
    """Host tensors, numbers that C would cut, and a scale per page without the other."""
    c = torch.zeros((2, 16, 2, 64), dtype=torch.float8_e4m3fn)
    i, n = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    x, w = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16), torch.zeros((2, 2, 16))
    for call in (lambda: sv.kv_weigh(x, c, i, n, w, w), lambda: sv.kv_select(w, None, i, n, n), lambda: sv.kv_move(c, c, i, n, i, i, n)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="layers"):
        sv.kv_select(torch.zeros((2, 2)), None, i, n, n)
    for wrong in (dict(first=-1), dict(recent=-1), dict(first=1 << 31), dict(recent=1 << 40)):
        with pytest.raises(ValueError, match="first and recent"):
            sv.kv_select(w, w.int(), i, n, n, **wrong)
