"""include/csa_draft.h without a GPU: exported symbols, struct layouts, and the refusals of bad host arguments,
each before any launch."""
import ctypes
import os
import re
import subprocess

import pytest

from sparse_attention_kv_e4m3_gb300 import build, draft, latent

HEADER = os.path.join(build.INCLUDE, "csa_draft.h")
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return draft.load()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(csa_[a-z_]+)\s*\(", text))
    assert names == {"csa_draft_abi_version", "csa_head_norm_rotate", "csa_latent_append", "csa_draft_attend", "csa_draft_attend_workspace_bytes",
                     "csa_draft_commit"}
    out = subprocess.run(["nm", "-D", "--defined-only", build.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(line.split()[-1] for line in out.splitlines() if line.strip())
    assert lib.csa_draft_abi_version() == 1


def test_limits_match_header():
    text = open(HEADER).read()
    got = {k: int(v) for k, v in re.findall(r"#define CSA_(\w+) (\d+)", text)}
    assert got["ROTATE_MAX_DIM"] == draft.ROTATE_MAX_DIM and got["ROTATE_MAX_ROPE"] == draft.ROTATE_MAX_ROPE
    assert got["ROTATE_MAX_HEADS"] == draft.ROTATE_MAX_HEADS
    assert got["DRAFT_MAX_WORDS"] == draft.MAX_WORDS and got["DRAFT_MAX_REQ"] == draft.MAX_REQ and got["COMMIT_MAX_REQ"] == draft.COMMIT_MAX_REQ
    assert draft.PAIRINGS == {"adjacent": got["PAIRS_ADJACENT"], "halves": got["PAIRS_HALVES"]}


@pytest.mark.parametrize("name,mirror", [
    ("csa_rotation", draft.RotationArgs), ("csa_heads", draft.HeadsArgs), ("csa_rotate_args", draft.RotateArgs), ("csa_append_args", draft.AppendArgs),
    ("csa_draft_attend_args", draft.DraftAttendArgs), ("csa_commit_args", draft.CommitArgs)])
def test_struct_layout_matches_header(tmp_path, name, mirror):
    fields = [f[0] for f in mirror._fields_]
    src = tmp_path / "layout.c"
    body = "".join(f'printf("{f} %zu\\n", offsetof({name}, {f}));' for f in fields)
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "csa_draft.h"\n'
                   'int main(void){' + body + f'printf("sizeof %zu\\n", sizeof({name}));return 0;}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", f"-I{build.INCLUDE}", "-o", str(exe), str(src)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for f in fields:
        assert int(got[f]) == getattr(mirror, f).offset, f
    assert int(got["sizeof"]) == ctypes.sizeof(mirror)


def _cache(**kw):
    d = dict(pages=0x10000, num_pages=8, page_stride_bytes=64 * 1152, rope_dim=64, record_format=0)
    d.update(kw)
    return latent.CacheArgs(**d)


CACHE_REFUSALS = [
    (dict(pages=0), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=1 << 31), INVALID),
    (dict(page_stride_bytes=64 * 1152 - 16), INVALID), (dict(page_stride_bytes=64 * 1152 + 8), ALIGNMENT),
    (dict(pages=0x10008), ALIGNMENT), (dict(rope_dim=32), UNSUPPORTED), (dict(record_format=2), UNSUPPORTED)]


def _rotation(**kw):
    d = dict(freq=0x7000, rope_dim=64, pairing=0, scale=1.0, reserved0=0)
    d.update(kw)
    return draft.RotationArgs(**d)


ROTATION_REFUSALS = [(dict(freq=0), INVALID), (dict(freq=0x7002), ALIGNMENT), (dict(pairing=2), INVALID), (dict(pairing=-1), INVALID),
                     (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(reserved0=1), INVALID), (dict(rope_dim=-2), INVALID)]


# ------------------------------------------------------------------ norm and rotation

def _heads(**kw):
    d = dict(x=0x10000, out=0x20000, weight=0x30000, x_row_stride=8 * 128, x_head_stride=128, out_row_stride=8 * 128, out_head_stride=128, heads=8,
             dim=128, norm=1, reserved0=0)
    d.update(kw)
    return draft.HeadsArgs(**d)


def _rotate(q=None, k=None, rotation=None, **kw):
    d = dict(q=_heads(**(q or {})), k=_heads(x=0x40000, out=0x50000, **{**dict(heads=1), **(k or {})}), n=3, pos=0x60000, rotation=_rotation(**(rotation or {})),
             dtype=1, out_dtype=1, rope_first=0, eps=1e-6, dev_status=0)
    d.update(kw)
    return draft.RotateArgs(**d)


HEADS_REFUSALS = [
    (dict(heads=-1), INVALID), (dict(heads=65537), UNSUPPORTED), (dict(dim=0), UNSUPPORTED), (dict(dim=132), UNSUPPORTED), (dict(dim=1032), UNSUPPORTED), (dict(dim=56), INVALID),
    (dict(norm=2), INVALID), (dict(reserved0=1), INVALID), (dict(weight=0x30008), ALIGNMENT)]


@pytest.mark.parametrize("change,want", [(dict(rotation=c), w) for c, w in ROTATION_REFUSALS] + [(dict(q=c), w) for c, w in HEADS_REFUSALS] + [
    (dict(k=c), w) for c, w in HEADS_REFUSALS] + [
    (dict(q=dict(x=0)), INVALID), (dict(q=dict(out=0)), INVALID), (dict(q=dict(x=0x10008)), ALIGNMENT), (dict(q=dict(out=0x20008)), ALIGNMENT),
    (dict(q=dict(x_head_stride=120)), INVALID), (dict(q=dict(out_head_stride=120)), INVALID), (dict(q=dict(x_row_stride=120)), INVALID),
    (dict(q=dict(out_row_stride=120)), INVALID), (dict(q=dict(x_head_stride=132)), ALIGNMENT), (dict(q=dict(out_row_stride=1028)), ALIGNMENT),
    (dict(q=dict(out=0x10000, out_row_stride=2048)), INVALID), (dict(q=dict(out=0x10000, out_head_stride=136)), INVALID),
    (dict(q=dict(out=0x10000), out_dtype=0), INVALID), (dict(q=dict(x_head_stride=132), dtype=0, n=0), OK),
    (dict(rotation=dict(rope_dim=272)), UNSUPPORTED), (dict(rotation=dict(rope_dim=24)), UNSUPPORTED), (dict(rotation=dict(rope_dim=144)), INVALID),
    (dict(pos=0), INVALID), (dict(pos=0x60002), ALIGNMENT), (dict(dev_status=0x1001), ALIGNMENT), (dict(n=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(out_dtype=-1), INVALID), (dict(rope_first=2), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID),
    (dict(n=0), OK), (dict(q=dict(heads=0, x=0, dim=7), k=dict(heads=0)), OK), (dict(n=0, q=dict(x=0)), OK), (dict(n=1 << 41), INVALID)])
def test_rotate_refusals(lib, change, want):
    assert lib.csa_head_norm_rotate(ctypes.byref(_rotate(**change)), None) == want


# ------------------------------------------------------------------ the rotating writer

def _append(cache=None, rotation=None, **kw):
    d = dict(cache=_cache(**(cache or {})), x=0x20000, x_stride=576, dtype=1, norm=1, n=3, slots=0x30000, pos=0x40000, rotation=_rotation(**(rotation or {})),
             weight=0x50000, eps=1e-6, reserved0=0, dev_status=0)
    d.update(kw)
    return draft.AppendArgs(**d)


@pytest.mark.parametrize("change,want", [(dict(cache=c), w) for c, w in CACHE_REFUSALS] + [(dict(rotation=c), w) for c, w in ROTATION_REFUSALS] + [
    (dict(x=0), INVALID), (dict(slots=0), INVALID), (dict(pos=0), INVALID), (dict(n=-1), INVALID), (dict(dtype=7), INVALID), (dict(norm=2), INVALID),
    (dict(reserved0=1), INVALID), (dict(x_stride=575), INVALID), (dict(x_stride=580), ALIGNMENT), (dict(x=0x20008), ALIGNMENT),
    (dict(slots=0x30004), ALIGNMENT), (dict(pos=0x40002), ALIGNMENT), (dict(weight=0x50004), ALIGNMENT), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID),
    (dict(rotation=dict(rope_dim=0)), INVALID), (dict(rotation=dict(rope_dim=32)), INVALID), (dict(n=0), OK), (dict(n=0, x=0), OK)])
def test_append_refusals(lib, change, want):
    assert lib.csa_latent_append(ctypes.byref(_append(**change)), None) == want


# ------------------------------------------------------------------ attention of drafts

def _attend(cache=None, **kw):
    d = dict(cache=_cache(**(cache or {})), q=0x20000, q_row_stride=16 * 576, q_head_stride=576, num_q=4, num_heads=16, page_table=0x30000, num_req=4,
             pt_stride=4, base_len=0x40000, row_start=0x50000, mask=0x60000, mask_stride=1, mask_words=1, scale=0.1, out=0x70000, lse=0x80000, dev_status=0)
    d.update(kw)
    return draft.DraftAttendArgs(**d)


@pytest.mark.parametrize("change,want", [(dict(cache=c), w) for c, w in CACHE_REFUSALS] + [
    (dict(num_heads=0), UNSUPPORTED), (dict(num_heads=129), UNSUPPORTED), (dict(num_req=65537), UNSUPPORTED), (dict(mask_words=17, mask_stride=17), UNSUPPORTED), (dict(q=0), INVALID),
    (dict(q=0x20008), ALIGNMENT), (dict(q_row_stride=16 * 576 + 4), ALIGNMENT), (dict(q_head_stride=575), INVALID), (dict(q_head_stride=580), ALIGNMENT),
    (dict(q_row_stride=568), INVALID), (dict(num_q=-1), INVALID), (dict(num_req=-1), INVALID), (dict(page_table=0), INVALID), (dict(pt_stride=0), INVALID),
    (dict(pt_stride=1 << 26), INVALID), (dict(pt_stride=(1 << 25) - 4), INVALID), (dict(base_len=0), INVALID), (dict(base_len=0x40002), ALIGNMENT), (dict(row_start=0), INVALID),
    (dict(row_start=0x50002), ALIGNMENT), (dict(mask=0x60004), ALIGNMENT), (dict(mask_words=0), INVALID), (dict(mask=0), INVALID),
    (dict(mask_words=2, mask_stride=1), INVALID), (dict(mask_words=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=NAN), INVALID), (dict(scale=2.0 ** 127), INVALID), (dict(out=0), INVALID), (dict(out=0x70008), ALIGNMENT), (dict(lse=0x80002), ALIGNMENT),
    (dict(dev_status=0x1001), ALIGNMENT), (dict(num_q=0), OK), (dict(num_req=0), OK)])
def test_attend_refusals(lib, change, want):
    assert lib.csa_draft_attend(ctypes.byref(_attend(**change)), 0x100000, 1 << 40, None) == want


def test_attend_workspace(lib):
    a = _attend()
    n = lib.csa_draft_attend_workspace_bytes(ctypes.byref(a))
    assert n > 0
    assert lib.csa_draft_attend(ctypes.byref(a), None, n, None) == WORKSPACE
    assert lib.csa_draft_attend(ctypes.byref(a), 0x100000, n - 1, None) == WORKSPACE
    assert lib.csa_draft_attend(ctypes.byref(a), 0x100010, n, None) == ALIGNMENT
    assert n == draft.draft_attend_workspace_bytes(4, 16, 4, 4)
    most = draft.draft_attend_workspace_bytes(1 << 20, 128, 1 << 10, 1 << 20)
    assert n <= most <= 90 << 20
    for bad in (dict(num_heads=200), dict(num_heads=0), dict(num_q=-1), dict(num_req=-1), dict(pt_stride=-1), dict(pt_stride=0), dict(pt_stride=1 << 26), dict(num_req=65537)):
        assert lib.csa_draft_attend_workspace_bytes(ctypes.byref(_attend(**bad))) == 0
    assert lib.csa_draft_attend_workspace_bytes(None) == 0


# ------------------------------------------------------------------ accepted drafts

def _commit(cache=None, **kw):
    d = dict(cache=_cache(**(cache or {})), layer_stride_bytes=8 * 64 * 1152, num_layers=3, num_req=4, page_table=0x20000, pt_stride=4, path_stride=5,
             base_len=0x30000, draft_len=0x40000, path=0x50000, path_len=0x60000, new_len=0x70000, freed=0x80000, room=7, n_freed=0x90000, dev_status=0)
    d.update(kw)
    return draft.CommitArgs(**d)


@pytest.mark.parametrize("change,want", [(dict(cache=c), w) for c, w in CACHE_REFUSALS] + [
    (dict(num_req=-1), INVALID), (dict(num_req=16385), UNSUPPORTED), (dict(num_layers=0), INVALID), (dict(layer_stride_bytes=64 * 1152 - 16), INVALID),
    (dict(layer_stride_bytes=64 * 1152 + 8), ALIGNMENT), (dict(page_table=0), INVALID), (dict(pt_stride=0), INVALID), (dict(pt_stride=1 << 26), INVALID),
    (dict(path_stride=-1), INVALID), (dict(base_len=0), INVALID), (dict(draft_len=0), INVALID), (dict(path=0), INVALID), (dict(path_len=0), INVALID),
    (dict(new_len=0), INVALID), (dict(new_len=0x30000), INVALID), (dict(new_len=0x40000), INVALID), (dict(new_len=0x60000), INVALID), (dict(freed=0), INVALID),
    (dict(room=-1), INVALID), (dict(n_freed=0), INVALID), (dict(path=0x50002), ALIGNMENT), (dict(new_len=0x70002), ALIGNMENT), (dict(freed=0x80001), ALIGNMENT),
    (dict(n_freed=0x90002), ALIGNMENT), (dict(dev_status=0x1002), ALIGNMENT), (dict(num_layers=1 << 30, num_req=16384), INVALID)])
def test_commit_refusals(lib, change, want):
    assert lib.csa_draft_commit(ctypes.byref(_commit(**change)), None) == want


def test_null_args(lib):
    assert lib.csa_head_norm_rotate(None, None) == INVALID
    assert lib.csa_latent_append(None, None) == INVALID
    assert lib.csa_draft_attend(None, 0x100000, 1 << 40, None) == INVALID
    assert lib.csa_draft_commit(None, None) == INVALID
