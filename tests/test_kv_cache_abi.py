"""Host-side checks of the cache's entry points (CPU only: nothing is launched)."""
import ctypes
import os
import re

import pytest

from precision_activation_quantization_b200 import pqg
from test_abi import FAKE, HEADER, host_only

INV, UNS, ALN = pqg.PQG_ERR_INVALID_ARG, pqg.PQG_ERR_UNSUPPORTED, pqg.PQG_ERR_ALIGNMENT


def at(i):
    return FAKE + (i << 34)


def cache(**kw):
    a = dict(k_codes=at(0), v_codes=at(1), k_scales=at(2), v_scales=at(3), global_scale=None,
             num_pages=8, page_size=64, kv_heads=2, head_dim=128, format=pqg.PQG_KV_MXFP4)
    a.update(kw)
    return pqg.pqg_kv_cache(**a)


def write(c=None, **kw):
    a = dict(k_ptr=at(4), v_ptr=at(5), slots_ptr=at(6), T=3, k_stride=256, v_stride=256,
             in_dtype=pqg.PQG_BF16, stream=None)
    a.update(kw)
    return pqg.pqg_kv_write(c or cache(), **a)


def read(c=None, **kw):
    a = dict(page_table_ptr=at(4), table_stride=3, max_pages=3, indptr_ptr=at(5), B=2,
             k_out_ptr=at(6), v_out_ptr=at(7), M=9, out_dtype=pqg.PQG_FP16, stream=None)
    a.update(kw)
    return pqg.pqg_kv_read(c or cache(), **a)


BAD_CACHES = [
    (dict(format=2), INV), (dict(format=-1), INV), (dict(page_size=0), INV),
    (dict(page_size=24), UNS), (dict(page_size=512), UNS), (dict(head_dim=-64), INV),
    (dict(head_dim=96), UNS), (dict(head_dim=512), UNS), (dict(kv_heads=0), INV),
    (dict(kv_heads=1025), INV), (dict(num_pages=0), INV), (dict(num_pages=1 << 25), INV),
    (dict(k_codes=0), INV), (dict(v_scales=0), INV), (dict(global_scale=at(8)), INV),
    (dict(format=pqg.PQG_KV_NVFP4), INV), (dict(v_codes=at(1) + 8), ALN),
    (dict(k_scales=at(2) + 4), ALN),
    (dict(format=pqg.PQG_KV_NVFP4, global_scale=at(8) + 2), ALN),
    (dict(v_codes=at(0) + 1024), INV), (dict(k_scales=at(1)), INV),
]


@host_only
@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(kw, status):
    before = pqg.pqg_launch_count()
    assert write(cache(**kw)) == status
    assert read(cache(**kw)) == status
    assert pqg.pqg_launch_count() == before


@host_only
@pytest.mark.parametrize("kw,status", [
    (dict(in_dtype=2), INV), (dict(T=-1), INV), (dict(T=1 << 31), INV), (dict(k_stride=240), INV),
    (dict(v_stride=255), INV), (dict(k_stride=264), ALN), (dict(k_stride=1 << 33), INV),
    (dict(k_ptr=0), INV), (dict(v_ptr=0), INV), (dict(slots_ptr=0), INV),
    (dict(k_ptr=at(4) + 16), ALN), (dict(v_ptr=at(5) + 2), ALN), (dict(slots_ptr=at(6) + 2), ALN),
    (dict(k_ptr=at(1)), INV), (dict(v_ptr=at(0) - 256), INV), (dict(slots_ptr=at(3)), INV),
])
def test_write_rejects(kw, status):
    before = pqg.pqg_launch_count()
    assert write(**kw) == status
    assert pqg.pqg_launch_count() == before


@host_only
@pytest.mark.parametrize("kw,status", [
    (dict(out_dtype=2), INV), (dict(M=-1), INV), (dict(M=1 << 31), INV), (dict(B=-1), INV),
    (dict(max_pages=0), INV), (dict(table_stride=2), INV), (dict(B=1 << 21), INV),
    (dict(page_table_ptr=0), INV), (dict(indptr_ptr=0), INV), (dict(k_out_ptr=0), INV),
    (dict(page_table_ptr=at(4) + 1), ALN), (dict(indptr_ptr=at(5) + 2), ALN),
    (dict(k_out_ptr=at(6) + 16), ALN), (dict(v_out_ptr=at(6) + 32), INV),
    (dict(k_out_ptr=at(4)), INV), (dict(v_out_ptr=at(5)), INV), (dict(v_out_ptr=at(2)), INV),
])
def test_read_rejects(kw, status):
    before = pqg.pqg_launch_count()
    assert read(**kw) == status
    assert pqg.pqg_launch_count() == before


@host_only
def test_nothing_to_do():
    before = pqg.pqg_launch_count()
    assert write(T=0, k_ptr=0, v_ptr=0, slots_ptr=0) == pqg.PQG_OK
    assert read(M=0, k_out_ptr=0, v_out_ptr=0) == pqg.PQG_OK
    assert read(B=0, page_table_ptr=0, indptr_ptr=0) == pqg.PQG_OK
    assert pqg.pqg_launch_count() == before


def test_a_missing_cache_is_refused():
    assert pqg.pqg_kv_write(None, 0, 0, 0, 0, 256, 256, 0, None) == INV


def test_struct_and_formats_match_the_header():
    text = open(HEADER).read()
    body = re.search(r"typedef struct pqg_kv_cache \{(.*?)\} pqg_kv_cache;", text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = re.findall(r"(\w+);", body)
    assert names == [n for n, _ in pqg.pqg_kv_cache._fields_]
    size = {"*": 8, "int64_t": 8, "int32_t": 4}
    declared = [size["*" if "*" in d else re.search(r"int\d+_t", d).group(0)]
                for d in body.split(";") if d.strip()]
    assert declared == [ctypes.sizeof(t) for _, t in pqg.pqg_kv_cache._fields_]
    for n in ("PQG_KV_MXFP4", "PQG_KV_NVFP4"):
        assert int(re.search(rf"\b{n}\s*=\s*(\d+)", text).group(1)) == getattr(pqg, n)
    assert os.path.exists(HEADER)


def attend(c=None, **kw):
    a = dict(q_ptr=at(4), q_stride=1024, page_table_ptr=at(5), table_stride=2, max_pages=2,
             seq_lens_ptr=at(6), B=2, q_len=1, q_heads=8, sm_scale=0.1, max_len=0, out_ptr=at(7),
             lse_ptr=at(8), workspace_ptr=None, workspace_bytes=0, in_dtype=pqg.PQG_BF16,
             stream=None)
    a.update(kw)
    return pqg.pqg_kv_attention(c or cache(), **a)


@host_only
@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_attention_bad_caches(kw, status):
    assert attend(cache(**kw)) == status
    assert pqg.pqg_kv_attention_workspace(cache(**kw), 3, 2, 1, 8, 0) == status


LONG = dict(max_pages=4096, table_stride=4096)      # 262144 keys: split, needs scratch


@host_only
@pytest.mark.parametrize("kw,status", [
    (dict(in_dtype=2), INV), (dict(B=-1), INV), (dict(B=1 << 21), INV), (dict(q_len=0), INV),
    (dict(q_len=1025), INV), (dict(q_heads=7), INV), (dict(q_heads=0), INV),
    (dict(q_heads=16386), INV), (dict(max_pages=0), INV), (dict(table_stride=1), INV),
    (dict(sm_scale=float("nan")), INV), (dict(sm_scale=float("inf")), INV),
    (dict(q_stride=1016), INV), (dict(q_stride=(1 << 30) + 8), INV), (dict(q_stride=1028), ALN),
    (dict(max_pages=1 << 31, table_stride=1 << 31), INV),
    (dict(B=1 << 20, max_pages=1 << 24, table_stride=1 << 24), INV),      # 2^44 pieces of keys
    (dict(q_ptr=0), INV), (dict(page_table_ptr=0), INV), (dict(seq_lens_ptr=0), INV),
    (dict(out_ptr=0), INV), (dict(q_ptr=at(4) + 8), ALN), (dict(out_ptr=at(7) + 8), ALN),
    (dict(lse_ptr=at(8) + 2), ALN), (dict(page_table_ptr=at(5) + 2), ALN),
    (dict(seq_lens_ptr=at(6) + 1), ALN), (dict(out_ptr=at(4)), INV), (dict(out_ptr=at(1)), INV),
    (dict(lse_ptr=at(7) + 64), INV), (dict(lse_ptr=at(6)), INV), (dict(out_ptr=at(5)), INV),
    (dict(LONG), INV),                                              # no scratch
    (dict(LONG, workspace_ptr=at(9), workspace_bytes=64), INV),     # too little
    (dict(LONG, workspace_ptr=at(9) + 8, workspace_bytes=1 << 30), ALN),
    (dict(LONG, workspace_ptr=at(7), workspace_bytes=1 << 30), INV),
    (dict(LONG, workspace_ptr=at(0), workspace_bytes=1 << 30), INV),
])
def test_attention_rejects(kw, status):
    before = pqg.pqg_launch_count()
    assert attend(**kw) == status
    assert pqg.pqg_launch_count() == before


@host_only
def test_attention_nothing_to_do_and_scratch():
    before = pqg.pqg_launch_count()
    assert attend(B=0, q_ptr=0, out_ptr=0, page_table_ptr=0, seq_lens_ptr=0) == pqg.PQG_OK
    assert pqg.pqg_launch_count() == before
    work = pqg.pqg_kv_attention_workspace
    assert work(cache(), 2, 2, 1, 8, 0) == 0                        # 128 keys: never divided
    assert work(cache(), 3, 2, 1, 8, 0) > 0
    assert work(cache(), 4096, 2, 1, 8, 100) > 0                    # the hint is no promise
    assert work(cache(), 4096, 0, 1, 8, 0) == 0
    assert work(cache(), 4096, 2, 1, 7, 0) == INV


@host_only
def test_attention_rejects_the_largest_sizes():
    """Every size at its own limit: counts of rows and pieces that pass 64 bits when multiplied."""
    c = cache(kv_heads=1024, num_pages=1)
    kw = dict(B=1 << 20, q_len=1024, q_heads=16384, q_stride=1 << 30, max_pages=1 << 30,
              table_stride=1 << 30)
    before = pqg.pqg_launch_count()
    assert attend(c, **kw) == INV
    assert pqg.pqg_kv_attention_workspace(c, 1 << 30, 1 << 20, 1024, 16384, 0) == INV
    assert pqg.pqg_launch_count() == before
