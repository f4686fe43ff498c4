"""CPU-only checks of the cache, tree-attention and head-norm entry points: what
they refuse is refused on the host before anything is launched, and the binding's
structures are the header's."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from sparse_latent_attention_indexer_gb300 import _abi
from sparse_latent_attention_indexer_gb300._abi import (DSA_BF16, DSA_E4M3, DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED,
                                                        DSA_ERR_WORKSPACE, DSA_F32, DSA_OK)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # an address that no check may dereference


def _seqs(T, S, P):
    return dsa.Seqs.from_lengths(T, S, P)


def _cache(dtype=DSA_BF16, **over):
    c = _abi.dsa_latent_cache(A, 576 if dtype != DSA_E4M3 else 512, A if dtype == DSA_E4M3 else None, A + 1024,
                              576 if dtype != DSA_E4M3 else 64, dtype, 4096)
    for k, v in over.items():
        setattr(c, k, v)
    return c


def _pages(**over):
    p = _abi.dsa_pages(A, 6, 4, 64, 64)
    for k, v in over.items():
        setattr(p, k, v)
    return p


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _write(cache=None, seqs=None, pages=None, x_dtype=DSA_BF16, c_kv=A, ld_c=512, k_pe=A, ld_x=64, d_c=512, d_r=64):
    seqs = seqs or _seqs([3, 0], [10, 5], [7, 5])
    return _abi.load().dsa_latent_cache_write(c_kv, ld_c, k_pe, ld_x, x_dtype, d_c, d_r, _ref(cache or _cache()),
                                              seqs.ref(), _ref(pages), None)


def _read(cache=None, seqs=None, pages=None, pos=None, out_dtype=DSA_BF16, c_kv=A, ld_c=512, k_pe=A, ld_x=64, d_c=512,
          d_r=64):
    seqs = seqs or _seqs([3, 0], [10, 5], [7, 5])
    return _abi.load().dsa_latent_cache_read(_ref(cache or _cache()), d_c, d_r, seqs.ref(), _ref(pages), pos, c_kv,
                                             ld_c, k_pe, ld_x, out_dtype, None)


BAD_CACHES = [
    (dict(kv=None), DSA_ERR_INVALID_ARG), (dict(kv=A + 8), DSA_ERR_INVALID_ARG), (dict(ld_kv=511), DSA_ERR_INVALID_ARG),
    (dict(ld_kv=516), DSA_ERR_INVALID_ARG), (dict(k_pe=None), DSA_ERR_INVALID_ARG), (dict(k_pe=A + 2), DSA_ERR_INVALID_ARG),
    (dict(ld_pe=63), DSA_ERR_INVALID_ARG), (dict(ld_pe=68), DSA_ERR_INVALID_ARG), (dict(rows=-1), DSA_ERR_INVALID_ARG),
    (dict(rows=14), DSA_ERR_INVALID_ARG),  # 15 contiguous tokens
    (dict(rows=2 ** 31 - 64), DSA_ERR_INVALID_ARG), (dict(dtype=7), DSA_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("call", [_write, _read])
@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_bad_caches_refused(call, over, status):
    assert call(cache=_cache(**over)) == status


@pytest.mark.parametrize("call", [_write, _read])
def test_moves_refuse_bad_arguments(call):
    dense = dict(c_kv=None), dict(k_pe=None), dict(c_kv=A + 1), dict(ld_c=511), dict(ld_x=63), dict(d_r=-1), dict(d_c=0)
    for over in dense:
        assert call(**over) == DSA_ERR_INVALID_ARG, over
    wide = _cache(ld_kv=2048, ld_pe=2048)
    assert call(cache=wide, d_c=1032, ld_c=2048) == DSA_ERR_UNSUPPORTED
    assert call(cache=wide, d_r=136, ld_x=2048) == DSA_ERR_UNSUPPORTED
    assert call(cache=_cache(DSA_E4M3), d_c=192) == DSA_ERR_UNSUPPORTED
    assert call(cache=_cache(DSA_E4M3, kv_scale=None)) == DSA_ERR_INVALID_ARG
    assert call(cache=_cache(DSA_E4M3, kv_scale=A + 2)) == DSA_ERR_INVALID_ARG
    assert call(seqs=_seqs([4], [10], [7])) == DSA_ERR_INVALID_ARG  # start_pos + T > S
    name = "x_dtype" if call is _write else "out_dtype"
    assert call(**{name: DSA_E4M3}) == DSA_ERR_UNSUPPORTED
    # no rows: every check that needs none passes and nothing is launched
    assert call(seqs=_seqs([0], [4], [4]), c_kv=None, k_pe=None) == DSA_OK
    assert dsa.last_launch_count() == 0


@pytest.mark.parametrize("call", [_write, _read])
def test_bad_pages_refused(call):
    good = dict(seqs=_seqs([3], [256], [250]))
    for over in (dict(page_size=0), dict(page_size=8), dict(page_size=24), dict(page_size=-16), dict(n_pages=-1),
                 dict(n_pages=65), dict(width=3), dict(width=-1), dict(ld_table=3), dict(block_table=None), dict(block_table=A + 2)):
        assert call(pages=_pages(**over), **good) == DSA_ERR_INVALID_ARG, over


def test_read_by_position_needs_a_table_of_the_whole_sequence():
    seqs = _seqs([3], [257], [10])  # 13 tokens are in reach by start_pos, 257 by position
    assert _read(pages=_pages(), seqs=seqs, pos=A) == DSA_ERR_INVALID_ARG
    assert _read(pages=_pages(), seqs=_seqs([3], [256], [10]), pos=A + 2) == DSA_ERR_INVALID_ARG


def _tree(cache=None, seqs=None, pages=None, dtype=DSA_BF16, dims=(128, 128, 64, 512, 128), mask=A, words=1, ws=A,
          ws_bytes=1 << 40, q=A, q_pe=A, W=A, out=A, lse=A):
    H, d_n, d_r, d_c, d_v = dims
    seqs = seqs or _seqs([3, 0], [10, 5], [7, 5])
    return _abi.load().dsa_tree_mla_fwd(q, q_pe, dtype, _ref(cache or _cache()), W, W, H, d_n, d_r, d_c, d_v, mask,
                                        words, seqs.ref(), _ref(pages), 0.1, out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_tree_refuses_bad_caches(over, status):
    assert _tree(cache=_cache(**over)) == status


def test_tree_refuses_bad_arguments():
    for over in (dict(q=None), dict(q_pe=None), dict(W=None), dict(out=None), dict(q=A + 8), dict(q_pe=A + 8),
                 dict(W=A + 8), dict(out=A + 8), dict(lse=A + 2), dict(mask=A + 4), dict(words=0)):
        assert _tree(**over) == DSA_ERR_INVALID_ARG, over
    assert _tree(seqs=_seqs([65], [70], [0])) == DSA_ERR_INVALID_ARG  # 65 nodes, one word of bits
    assert _tree(seqs=_seqs([65], [70], [0]), words=2, ws=None) == DSA_ERR_WORKSPACE
    assert _tree(ws=None) == DSA_ERR_WORKSPACE
    assert _tree(ws=A + 128) == DSA_ERR_WORKSPACE
    assert _tree(ws_bytes=255) == DSA_ERR_WORKSPACE
    assert _tree(dtype=DSA_E4M3) == DSA_ERR_UNSUPPORTED
    assert _tree(dtype=DSA_F32) == DSA_ERR_UNSUPPORTED                          # fp32 queries, bf16 cache
    assert _tree(cache=_cache(DSA_F32)) == DSA_ERR_UNSUPPORTED                  # and the other way round
    assert _tree(dims=(257, 128, 64, 512, 128)) == DSA_ERR_UNSUPPORTED
    assert _tree(dims=(0, 128, 64, 512, 128)) == DSA_ERR_INVALID_ARG
    assert _tree(pages=_pages(width=0)) == DSA_ERR_INVALID_ARG
    assert _tree(seqs=_seqs([0], [4], [4]), q=None, out=None, ws=None) == DSA_OK
    assert dsa.last_launch_count() == 0


def test_tree_workspace_is_what_the_call_asks_for():
    lib = _abi.load()
    for T, S, P in (([1], [778], [777]), ([32] * 16, [9000] * 16, [8968] * 16), ([7, 0, 301], [20, 9, 5302], [13, 9, 5001])):
        s = _seqs(T, S, P)
        for H in (16, 128):
            need = lib.dsa_tree_mla_workspace_size(DSA_BF16, H, 128, 64, 512, 128, s.ref())
            assert need > 0 and need % 256 == 0
            c = _cache(rows=1 << 20)
            assert _tree(cache=c, seqs=s, dims=(H, 128, 64, 512, 128), words=5, ws_bytes=need - 1) == DSA_ERR_WORKSPACE
    assert lib.dsa_tree_mla_workspace_size(DSA_E4M3, 128, 128, 64, 512, 128, s.ref()) == 0
    assert lib.dsa_tree_mla_workspace_size(DSA_BF16, 128, 128, 64, 512, 128, _seqs([4], [3], [0]).ref()) == 0


def _heads(**over):
    h = _abi.dsa_heads(A, 1024, 128, 8, _abi.DSA_NORM_RMS, A, None, A + 4096, 1024, 128, None, 0, 0)
    for k, v in over.items():
        setattr(h, k, v)
    return h


def _norm(q=None, k=None, x=DSA_BF16, y=DSA_BF16, D=128, d_r=64, rope=0, eps=1e-6, cos=A, sin=A, n_pos=100, pos=None,
          seqs=None):
    seqs = seqs or _seqs([3], [10], [7])
    return _abi.load().dsa_head_norm_rope(_ref(q), _ref(k), x, y, D, d_r, 0, rope, eps, cos, sin, n_pos, pos,
                                          seqs.ref(), None)


def test_head_norm_refuses_bad_arguments():
    for over in (dict(x=None), dict(y=None), dict(x=A + 1), dict(y=A + 1), dict(gain=A + 2), dict(bias=A + 2),
                 dict(n_heads=-1), dict(y_pe=A + 1), dict(y=A, ld_y=2048), dict(y=A, hd_y=256),
                 dict(y=A, y_pe=A + 4096)):
        for place in ("q", "k"):
            assert _norm(**{place: _heads(**over)}) == DSA_ERR_INVALID_ARG, over
    good = _heads()
    for over in (dict(d_r=63), dict(d_r=130), dict(d_r=-2), dict(D=0), dict(cos=None), dict(sin=None), dict(n_pos=9),
                 dict(pos=A + 2), dict(eps=-1.0), dict(eps=float("nan")), dict(cos=A + 2)):
        assert _norm(q=good, **over) == DSA_ERR_INVALID_ARG, over
    assert _norm(q=_heads(y=A), y=DSA_F32) == DSA_ERR_INVALID_ARG  # in place across types
    assert _norm(q=_heads(y_pe=A), d_r=0) == DSA_ERR_INVALID_ARG
    for over in (dict(D=513), dict(x=DSA_E4M3), dict(y=DSA_E4M3), dict(rope=2)):
        assert _norm(q=good, **over) == DSA_ERR_UNSUPPORTED, over
    assert _norm(q=_heads(norm=3)) == DSA_ERR_UNSUPPORTED
    assert _norm() == DSA_OK and _norm(q=_heads(n_heads=0, x=None)) == DSA_OK  # no heads: nothing to do
    assert _norm(q=_heads(x=None, y=None), seqs=_seqs([0], [4], [4])) == DSA_OK
    assert dsa.last_launch_count() == 0


def test_binding_refuses_what_does_not_fit():
    cpu = dsa.LatentCache(torch.zeros(32, 512), torch.zeros(32, 64))
    seqs = _seqs([2], [8], [6])
    with pytest.raises(ValueError, match="CUDA tensor"):
        dsa.dsa_latent_cache_write(torch.zeros(2, 512), torch.zeros(2, 64), cpu, seqs)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dsa.dsa_latent_cache_read(cpu, seqs)
    with pytest.raises(ValueError, match="kv_scale"):
        dsa.LatentCache(torch.zeros(4, 512, dtype=torch.uint8), torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="kv_scale"):
        dsa.LatentCache(torch.zeros(4, 512), torch.zeros(4, 64), torch.zeros(4, 4))
    with pytest.raises(ValueError, match="k_pe is"):
        dsa.LatentCache(torch.zeros(4, 512).bfloat16(), torch.zeros(4, 64))
    with pytest.raises(ValueError, match="expected"):
        dsa.LatentCache(torch.zeros(4, 512), torch.zeros(5, 64))
    with pytest.raises(ValueError, match="contiguous rows"):
        dsa.LatentCache(torch.zeros(512, 4).t(), torch.zeros(4, 64))
    with pytest.raises(ValueError, match="int32"):
        dsa.Pages(torch.zeros(1, 4), 64, 4)
    pages = dsa.Pages(torch.zeros(1, 2, dtype=torch.int32), 16, 4)
    with pytest.raises(ValueError, match="rows for 2"):
        pages.ref("f", _seqs([1, 1], [4, 4], [3, 3]))
    with pytest.raises(ValueError, match="norm must be"):
        dsa.Heads(torch.zeros(1, 1, 8), norm="batch")
    with pytest.raises(ValueError, match="neither"):
        dsa.dsa_head_norm_rope(None, None, torch.zeros(4, 4), torch.zeros(4, 4), seqs)


def test_structures_match_the_header(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    structs = [_abi.dsa_pages, _abi.dsa_latent_cache, _abi.dsa_heads]
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "dsa.h"', "int main(void) {"]
    consts = re.findall(r"#define (DSA_(?:NORM|ROPE)_[A-Z]+)\s", open(os.path.join(ROOT, "include", "dsa.h")).read())
    assert len(consts) == 5
    lines += [f'    printf("{c} value %d\\n", {c});' for c in consts]
    for st in structs:
        n = st.__name__
        lines.append(f'    printf("{n} size %zu\\n", sizeof({n}));')
        lines += [f'    printf("{n} {f} %zu\\n", offsetof({n}, {f}));' for f, _ in st._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["    return 0;", "}"]) + "\n")
    subprocess.run([gcc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = {}
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        n, f, v = line.split()
        got[(n, f)] = int(v)
    for c in consts:
        assert got[(c, "value")] == getattr(_abi, c)
    for st in structs:
        assert got[(st.__name__, "size")] == ctypes.sizeof(st)
        for f, _ in st._fields_:
            assert got[(st.__name__, f)] == getattr(st, f).offset


def test_tree_refuses_positions_at_the_end_of_32_bits():
    """Token numbers are counted in tiles beyond the last one."""
    end = 2 ** 31 - 1
    pages = _pages(page_size=1 << 20, n_pages=0, width=1 << 12, ld_table=1 << 12)
    assert _tree(seqs=_seqs([3], [end], [end - 3]), pages=pages) == DSA_ERR_UNSUPPORTED
    assert _tree(seqs=_seqs([3], [end], [end - 130]), pages=pages, ws=None) in (DSA_ERR_UNSUPPORTED, DSA_ERR_WORKSPACE)
