"""include/csa_latent.h without a GPU: exported symbols, struct layouts, record sizes and the
refusals of bad host arguments, each before any launch."""
import ctypes
import os
import re
import subprocess

import pytest

from sparse_attention_kv_e4m3_gb300 import build, latent, native

HEADER = os.path.join(build.INCLUDE, "csa_latent.h")
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    build.build()
    return latent.load()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(csa_[a-z_]+)\s*\(", text)))
    assert {"csa_build_tables", "csa_latent_write", "csa_latent_read", "csa_latent_attend", "csa_latent_prefill",
            "csa_latent_attend_workspace_bytes", "csa_latent_record_bytes", "csa_latent_abi_version"} == set(names)
    out = subprocess.run(["nm", "-D", "--defined-only", build.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = set(line.split()[-1] for line in out.splitlines() if line.strip())
    assert set(names) <= exported
    assert lib.csa_latent_abi_version() == 1


@pytest.mark.parametrize("name,mirror", [
    ("csa_latent_cache", latent.CacheArgs), ("csa_tables_args", latent.TablesArgs),
    ("csa_latent_write_args", latent.LatentWriteArgs), ("csa_latent_read_args", latent.LatentReadArgs),
    ("csa_latent_attend_args", latent.AttendArgs), ("csa_latent_prefill_args", latent.PrefillArgs)])
def test_struct_layout_matches_header(tmp_path, name, mirror):
    fields = [f[0] for f in mirror._fields_]
    src = tmp_path / "layout.c"
    body = "".join(f'printf("{f} %zu\\n", offsetof({name}, {f}));' for f in fields)
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "csa_latent.h"\n'
                   'int main(void){' + body + f'printf("sizeof %zu\\n", sizeof({name}));return 0;}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", f"-I{build.INCLUDE}", "-o", str(exe), str(src)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for f in fields:
        assert int(got[f]) == getattr(mirror, f).offset, f
    assert int(got["sizeof"]) == ctypes.sizeof(mirror)


def test_record_bytes(lib):
    f = lib.csa_latent_record_bytes
    assert [f(0, 0), f(0, 64), f(1, 0), f(1, 64)] == [1024, 1152, 272, 400]
    assert [f(2, 0), f(-1, 64), f(0, 32), f(1, -64)] == [0, 0, 0, 0]
    with pytest.raises(ValueError):
        latent.record_bytes("fp8", 64)


def _cache(**kw):
    d = dict(pages=0x10000, num_pages=8, page_stride_bytes=64 * 1152, rope_dim=64, record_format=0)
    d.update(kw)
    return latent.CacheArgs(**d)


CACHE_REFUSALS = [
    (dict(pages=0), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=1 << 31), INVALID),
    (dict(page_stride_bytes=64 * 1152 - 16), INVALID), (dict(page_stride_bytes=64 * 1152 + 8), ALIGNMENT),
    (dict(pages=0x10008), ALIGNMENT), (dict(rope_dim=32), UNSUPPORTED), (dict(record_format=2), UNSUPPORTED)]


def _tables(**kw):
    d = dict(old_len=0x1000, new_len=0x2000, num_req=4, pt_stride=8, page_table=0x3000, free_pages=0x4000, n_free=5,
             n_rows=7, row_req=0x5000, row_pos=0x6000, row_len=0x7000, row_slot=0x8000, row_start=0x9000,
             kv_start=0xA000, taken=0xB000, dev_status=0)
    d.update(kw)
    return latent.TablesArgs(**d)


@pytest.mark.parametrize("change,want", [
    (dict(num_req=-1), INVALID), (dict(num_req=16385), UNSUPPORTED), (dict(old_len=0), INVALID), (dict(new_len=0), INVALID),
    (dict(page_table=0), INVALID), (dict(pt_stride=0), INVALID), (dict(pt_stride=1 << 26), INVALID), (dict(free_pages=0), INVALID),
    (dict(n_free=-1), INVALID), (dict(n_rows=-1), INVALID), (dict(row_req=0), INVALID), (dict(row_pos=0), INVALID),
    (dict(row_len=0), INVALID), (dict(row_slot=0), INVALID), (dict(row_start=0), INVALID), (dict(kv_start=0), INVALID),
    (dict(taken=0), INVALID), (dict(row_slot=0x8004), ALIGNMENT), (dict(old_len=0x1002), ALIGNMENT), (dict(dev_status=0xC001), ALIGNMENT)])
def test_tables_refusals(lib, change, want):
    assert lib.csa_build_tables(ctypes.byref(_tables(**change)), None) == want


def _write(cache=None, **kw):
    d = dict(cache=_cache(**(cache or {})), x=0x20000, x_stride=576, dtype=native.KEYS_BF16, reserved0=0, n=3, slots=0x30000, dev_status=0)
    d.update(kw)
    return latent.LatentWriteArgs(**d)


@pytest.mark.parametrize("change,want", [(dict(cache=c), w) for c, w in CACHE_REFUSALS] + [
    (dict(x=0), INVALID), (dict(slots=0), INVALID), (dict(n=-1), INVALID), (dict(dtype=7), INVALID), (dict(reserved0=1), INVALID),
    (dict(x_stride=575), INVALID), (dict(x_stride=580), ALIGNMENT), (dict(x=0x20008), ALIGNMENT), (dict(slots=0x30004), ALIGNMENT),
    (dict(n=0), OK), (dict(n=0, x=0), OK)])
def test_write_refusals(lib, change, want):
    assert lib.csa_latent_write(ctypes.byref(_write(**change)), None) == want


def _read(cache=None, **kw):
    d = dict(cache=_cache(**(cache or {})), page_table=0x20000, num_req=2, pt_stride=4, kv_start=0x30000, n_rows=9, out=0x40000, dev_status=0)
    d.update(kw)
    return latent.LatentReadArgs(**d)


@pytest.mark.parametrize("change,want", [(dict(cache=c), w) for c, w in CACHE_REFUSALS] + [
    (dict(page_table=0), INVALID), (dict(kv_start=0), INVALID), (dict(out=0), INVALID), (dict(n_rows=-1), INVALID),
    (dict(num_req=-1), INVALID), (dict(pt_stride=0), INVALID), (dict(out=0x40008), ALIGNMENT), (dict(kv_start=0x30002), ALIGNMENT),
    (dict(n_rows=0), OK), (dict(num_req=0), OK)])
def test_read_refusals(lib, change, want):
    assert lib.csa_latent_read(ctypes.byref(_read(**change)), None) == want


def _attend(cache=None, **kw):
    d = dict(cache=_cache(**(cache or {})), q=0x20000, q_row_stride=16 * 576, q_head_stride=576, num_q=4, num_heads=16,
             page_table=0x30000, num_req=4, pt_stride=4, row_req=0, row_len=0x40000, idx=0, idx_stride=0, top=0, scale=0.1,
             out=0x50000, lse=0x60000, dev_status=0)
    d.update(kw)
    return latent.AttendArgs(**d)


@pytest.mark.parametrize("change,want", [(dict(cache=c), w) for c, w in CACHE_REFUSALS] + [
    (dict(num_heads=0), UNSUPPORTED), (dict(num_heads=129), UNSUPPORTED), (dict(q=0), INVALID), (dict(q=0x20008), ALIGNMENT),
    (dict(q_row_stride=16 * 576 + 4), ALIGNMENT), (dict(q_head_stride=575), INVALID), (dict(q_head_stride=580), ALIGNMENT),
    (dict(num_q=-1), INVALID), (dict(num_req=3), INVALID), (dict(page_table=0), INVALID), (dict(pt_stride=0), INVALID),
    (dict(row_len=0), INVALID), (dict(row_len=0x40002), ALIGNMENT), (dict(top=5), INVALID), (dict(idx=0x70000), INVALID),
    (dict(idx=0x70000, top=8, idx_stride=7), INVALID), (dict(idx=0x70002, top=8, idx_stride=8), ALIGNMENT),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(out=0), INVALID), (dict(out=0x50008), ALIGNMENT), (dict(lse=0x60002), ALIGNMENT), (dict(num_q=0), OK)])
def test_attend_refusals(lib, change, want):
    a = _attend(**change)
    n = lib.csa_latent_attend_workspace_bytes(ctypes.byref(a))
    assert lib.csa_latent_attend(ctypes.byref(a), 0x100000, max(n, 1 << 30), None) == want


def test_attend_workspace_refusals(lib):
    a = _attend()
    n = lib.csa_latent_attend_workspace_bytes(ctypes.byref(a))
    assert n > 0
    assert lib.csa_latent_attend(ctypes.byref(a), None, n, None) == WORKSPACE
    assert lib.csa_latent_attend(ctypes.byref(a), 0x100000, n - 1, None) == WORKSPACE
    assert lib.csa_latent_attend(ctypes.byref(a), 0x100008, n, None) == ALIGNMENT
    assert lib.csa_latent_attend_workspace_bytes(ctypes.byref(_attend(num_heads=200))) == 0
    assert lib.csa_latent_attend_workspace_bytes(ctypes.byref(_attend(num_q=-1))) == 0
    assert lib.csa_latent_attend_workspace_bytes(None) == 0
    assert lib.csa_latent_attend(None, 0x100000, n, None) == INVALID


def _prefill(**kw):
    d = dict(q=0x10000, k_nope=0x20000, k_rope=0x30000, v=0x40000, q_row_stride=4 * 192, q_head_stride=192, k_row_stride=4 * 256,
             k_head_stride=256, rope_row_stride=576, v_row_stride=4 * 256, v_head_stride=256, total_q=10, total_k=20, q_start=0x50000,
             kv_start=0x60000, num_req=2, num_heads=4, causal=1, scale=0.1, out=0x70000, lse=0x80000, dev_status=0)
    d.update(kw)
    return latent.PrefillArgs(**d)


@pytest.mark.parametrize("change,want", [
    (dict(q=0), INVALID), (dict(k_nope=0), INVALID), (dict(k_rope=0), INVALID), (dict(v=0), INVALID), (dict(q_start=0), INVALID),
    (dict(kv_start=0), INVALID), (dict(out=0), INVALID), (dict(total_q=-1), INVALID), (dict(total_k=-1), INVALID), (dict(num_req=-1), INVALID),
    (dict(num_heads=0), UNSUPPORTED), (dict(causal=2), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(q=0x10008), ALIGNMENT), (dict(v=0x40008), ALIGNMENT), (dict(k_row_stride=1028), ALIGNMENT), (dict(rope_row_stride=0), INVALID),
    (dict(v_head_stride=257), ALIGNMENT), (dict(q_start=0x50002), ALIGNMENT), (dict(total_q=1 << 31), INVALID),
    (dict(total_q=0), OK), (dict(num_req=0), OK)])
def test_prefill_refusals(lib, change, want):
    assert lib.csa_latent_prefill(ctypes.byref(_prefill(**change)), None) == want


def test_null_args(lib):
    assert lib.csa_build_tables(None, None) == INVALID
    assert lib.csa_latent_write(None, None) == INVALID
    assert lib.csa_latent_read(None, None) == INVALID
    assert lib.csa_latent_prefill(None, None) == INVALID


def test_binding_refuses_host_tensors():
    import torch

    x = torch.zeros(4, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        latent.LatentCache(torch.zeros(2, 64 * 1152, dtype=torch.uint8))
    ints = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        latent.csa_build_tables(ints, ints, ints.reshape(3, 1), ints, 4)
    with pytest.raises(ValueError):
        latent.csa_latent_prefill(x.reshape(4, 3, 192), x, x, x, ints, ints, scale=1.0)
