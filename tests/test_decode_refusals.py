"""What the decode-step operators refuse before they touch the device (CPU only): the C entry points' status
codes, the header's declarations, and the binding's checks."""
import ctypes
import os

import pytest
import torch

import speculative_decoding_rejection_verify_gb300 as sv
from speculative_decoding_rejection_verify_gb300 import _build, decode
from test_abi import INCLUDE, declared_functions

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sv.load()


def heads(**kw):
    a = dict(data=4096, row_stride=4096, token_stride=1024, head_stride=128)
    a.update(kw)
    return ctypes.byref(decode.HeadsStruct(*a.values()))


def cache(**kw):
    a = dict(k=4096, v=4096, layer_stride=0, page_stride=16 * 1024, slot_stride=1024, head_stride=128, layers=1,
             num_pages=4, page_size=16, heads=8, head_dim=128, dtype=sv.DTYPE_BF16, k_scale=None, v_scale=None)
    a.update(kw)
    return ctypes.byref(decode.CacheStruct(*a.values()))


def batch(**kw):
    a = dict(pages=4096, ctx_len=4096, t_per_row=None, B=1, T=2, max_pages=3)
    a.update(kw)
    return ctypes.byref(decode.BatchStruct(*a.values()))


BAD_CACHES = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=4104), INVALID), (dict(v=4098), INVALID),
              (dict(layers=0), INVALID), (dict(num_pages=-1), INVALID), (dict(heads=0), INVALID), (dict(page_size=0), INVALID),
              (dict(slot_stride=1020), INVALID), (dict(page_stride=-16), INVALID), (dict(head_stride=4), INVALID),
              (dict(k_scale=4096), INVALID), (dict(v_scale=4096), INVALID), (dict(dtype=sv.DTYPE_F32), UNSUPPORTED),
              (dict(dtype=7), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED),
              (dict(page_size=4), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED), (dict(page_size=8192), UNSUPPORTED),
              (dict(dtype=decode.DTYPE_E4M3, head_stride=72), INVALID)]
BAD_BATCHES = [(dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(pages=None), INVALID),
               (dict(ctx_len=None), INVALID), (dict(max_pages=2 ** 26 + 1), UNSUPPORTED)]


def append(lib, q=True, k=None, v=None, o=True, n=8, c=None, b=None, r=None):
    h = lambda x: heads() if x is True or x is None else x or None  # noqa: E731
    return lib.spec_kv_append(h(q) if q else None, h(k), h(v), h(o) if o else None, n, c or cache(), b or batch(), r, None, None)


def attend(lib, q=None, o=None, n=8, c=None, b=None, scale=0.1, ws=4096, wsb=1 << 30):
    return lib.spec_paged_attention(q or heads(), o or heads(), n, c or cache(), b or batch(), None, scale, ws, wsb, None)


def keep(lib, c=None, b=None, path=4096, n=4096, m=3):
    return lib.spec_kv_keep(c or cache(), b or batch(), path, n, m, None)


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches(lib, change, status):
    c = cache(**change)
    assert append(lib, c=c) == status
    assert attend(lib, c=c) == status
    if "scale" not in next(iter(change)):
        assert keep(lib, c=c) == status


@pytest.mark.parametrize("change,status", BAD_BATCHES)
def test_bad_batches(lib, change, status):
    b = batch(**change)
    assert append(lib, b=b) == status
    assert attend(lib, b=b) == status
    if "T" not in change:
        assert keep(lib, b=b) == status


def test_missing_structs(lib):
    assert lib.spec_kv_append(None, heads(), heads(), None, 0, None, batch(), None, None, None) == INVALID
    assert lib.spec_kv_append(None, heads(), heads(), None, 0, cache(), None, None, None, None) == INVALID
    assert lib.spec_kv_append(None, None, heads(), None, 0, cache(), batch(), None, None, None) == INVALID
    assert lib.spec_paged_attention(None, heads(), 8, cache(), batch(), None, 1.0, 4096, 1 << 30, None) == INVALID
    assert lib.spec_paged_attention(heads(), None, 8, cache(), batch(), None, 1.0, 4096, 1 << 30, None) == INVALID
    assert lib.spec_kv_keep(None, batch(), 4096, 4096, 1, None) == INVALID
    assert lib.spec_kv_keep(cache(), None, 4096, 4096, 1, None) == INVALID
    assert lib.spec_process_logits(4096, 4096, None, 1, 1, 8, 0, None) == INVALID


def test_append_arguments(lib):
    assert append(lib, n=-1) == INVALID
    assert append(lib, n=0) == INVALID            # q given, no heads
    assert append(lib, q=False) == INVALID        # heads, no q
    assert append(lib, o=False) == INVALID
    assert append(lib, k=heads(data=None)) == INVALID
    assert append(lib, v=heads(data=4100)) == INVALID
    assert append(lib, k=heads(token_stride=1022)) == INVALID
    R = lambda *a: ctypes.byref(decode.RotaryStruct(*a))  # noqa: E731
    for r in (R(4096, 4096, None, 24, 9, 0), R(4096, 4096, None, -16, 9, 0), R(4096, 4096, None, 144, 9, 0),
              R(None, 4096, None, 64, 9, 0), R(4096, None, None, 64, 9, 0), R(4096, 4100, None, 64, 9, 0),
              R(4096, 4096, None, 64, 0, 0)):
        assert append(lib, r=r) == INVALID
    assert append(lib, b=batch(B=0)) == OK        # nothing to do
    assert append(lib, b=batch(T=0)) == OK
    assert append(lib, b=batch(T=2 ** 30 + 1)) == UNSUPPORTED


def test_attention_arguments(lib):
    assert attend(lib, n=0) == INVALID
    assert attend(lib, n=12) == INVALID           # not a multiple of the kv heads
    assert attend(lib, scale=float("nan")) == INVALID
    assert attend(lib, scale=float("inf")) == INVALID
    assert attend(lib, q=heads(data=4098)) == INVALID
    assert attend(lib, o=heads(row_stride=4)) == INVALID
    assert attend(lib, b=batch(T=65)) == UNSUPPORTED
    assert attend(lib, n=8 * 129) == UNSUPPORTED
    assert attend(lib, ws=None) == WORKSPACE
    assert attend(lib, ws=4096 + 128) == WORKSPACE
    assert attend(lib, wsb=16) == WORKSPACE
    assert attend(lib, b=batch(B=0)) == OK
    assert attend(lib, b=batch(T=0)) == OK
    size = lib.spec_paged_attention_workspace_bytes
    assert size(8, 5, 32, 8, 128) % 256 == 0 and size(8, 5, 32, 8, 128) > 0
    for bad in ((-1, 5, 32, 8, 128), (8, 65, 32, 8, 128), (8, 5, 31, 8, 128), (8, 5, 0, 8, 128), (8, 5, 32, 0, 128),
                (8, 5, 32, 8, 80), (8, 5, 258, 2, 64)):
        assert size(*bad) == 0


def test_keep_arguments(lib):
    assert keep(lib, m=-1) == INVALID
    assert keep(lib, path=None) == INVALID
    assert keep(lib, n=None) == INVALID
    assert keep(lib, m=0, path=None, n=None) == OK
    assert keep(lib, b=batch(B=0)) == OK


def rules(**kw):
    r = decode.RulesStruct()
    for k, x in kw.items():
        setattr(r, k, x)
    return ctypes.byref(r)


def shape_logits(lib, r=None, z=4096, o=4096, B=1, T=1, V=64, dtype=0):
    return lib.spec_process_logits(z, o, r or rules(), B, T, V, dtype, None)


def test_logits_arguments(lib):
    assert shape_logits(lib, B=-1) == INVALID
    assert shape_logits(lib, T=-1) == INVALID
    assert shape_logits(lib, V=0) == INVALID
    assert shape_logits(lib, z=None) == INVALID
    assert shape_logits(lib, o=None) == INVALID
    assert shape_logits(lib, z=4098) == INVALID
    assert shape_logits(lib, o=4097, dtype=1) == INVALID
    assert shape_logits(lib, dtype=decode.DTYPE_E4M3) == UNSUPPORTED
    assert shape_logits(lib, V=sv.MAX_V + 1) == UNSUPPORTED
    assert shape_logits(lib, B=65536) == UNSUPPORTED
    assert shape_logits(lib, T=65) == UNSUPPORTED
    assert shape_logits(lib, rules(history_stride=-1)) == INVALID
    assert shape_logits(lib, rules(history=4096, history_stride=9)) == INVALID      # no lengths
    assert shape_logits(lib, rules(bias_n=3, bias=4096)) == INVALID
    assert shape_logits(lib, rules(bias_n=3, bias_ids=4096)) == INVALID
    assert shape_logits(lib, rules(bias_n=-1)) == INVALID
    assert shape_logits(lib, rules(bias_n=decode.MAX_BIAS + 1, bias=4096, bias_ids=4096)) == UNSUPPORTED
    assert shape_logits(lib, rules(history_stride=decode.MAX_HISTORY + 1)) == UNSUPPORTED
    assert shape_logits(lib, B=0) == OK
    assert shape_logits(lib, T=0) == OK


def test_header_and_binding_agree():
    header = os.path.join(INCLUDE, "spec_decode.h")
    assert set(declared_functions(header)) == set(sv.DECODE_EXPORTS)
    text = open(header).read()
    for name, value in (("MAX_BATCH", decode.MAX_BATCH), ("MAX_NEW", decode.MAX_NEW), ("MAX_GROUP", decode.MAX_GROUP), ("MAX_PAGE", decode.MAX_PAGE),
                        ("MAX_HISTORY", decode.MAX_HISTORY), ("MAX_BIAS", decode.MAX_BIAS),
                        ("FLAG_BAD_SLOT", decode.FLAG_BAD_SLOT), ("FLAG_BAD_POSITION", decode.FLAG_BAD_POSITION)):
        assert f"#define SPEC_{name} {value} " in text, name


def test_structs_match_the_header(tmp_path):
    """The binding's struct sizes and fields' offsets are the C compiler's, and its packed bytes lie as they do."""
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    pairs = (("spec_heads_t", decode.HeadsStruct), ("spec_kv_cache_t", decode.CacheStruct),
             ("spec_decode_batch_t", decode.BatchStruct), ("spec_rotary_t", decode.RotaryStruct),
             ("spec_logit_rules_t", decode.RulesStruct))
    body = "".join(f'printf("%zu\\n", sizeof({n}));' + "".join(f'printf("%zu\\n", offsetof({n}, {f[0]}));' for f in s._fields_)
                   for n, s in pairs)
    src = tmp_path / "s.c"
    src.write_text('#include "spec_decode.h"\n#include <stdio.h>\nint main(void) {' + body + "return 0;}\n")
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", INCLUDE, str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    want = [n for _, s in pairs for n in [ctypes.sizeof(s)] + [getattr(s, f[0]).offset for f in s._fields_]]
    assert got == want
    for pack, cls in ((decode._pack_heads, decode.HeadsStruct), (decode._pack_cache, decode.CacheStruct),
                      (decode._pack_batch, decode.BatchStruct), (decode._pack_rotary, decode.RotaryStruct),
                      (decode._pack_rules, decode.RulesStruct)):
        values = list(range(1, len(cls._fields_) + 1))
        s = cls.from_buffer_copy(pack(*values))
        assert [getattr(s, f[0]) for f in cls._fields_] == values


def test_binding_refuses_host_tensors_and_wrong_types(lib):
    c = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 2), dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    x = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: sv.paged_attention(x, c, c, i, n), lambda: sv.kv_append(x, x, x, c, c, i, n),
                 lambda: sv.kv_keep(c, c, i, n, i, n), lambda: sv.process_logits(torch.zeros((1, 1, 8)))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match=r"\[B, T, V\]"):
        sv.process_logits(torch.zeros((1, 8)))
