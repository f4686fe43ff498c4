"""CPU-only checks of calls of the cache, tree-attention and head-norm entry points that are refused, and of the
batch description (see test_cache_tree_host for the others)."""
import array
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from sparse_latent_attention_indexer_gb300._abi import DSA_ERR_UNSUPPORTED
from tests.test_cache_tree_host import _heads, _norm, _pages, _read, _seqs, _write


def test_a_mask_without_words_is_no_chain(monkeypatch):
    """The address of an empty tensor is NULL, which the library takes for a chain: the binding refuses it."""
    monkeypatch.setattr(dsa, "_on_one_device", lambda fn, tensors: 0)  # host tensors stand in: nothing is launched
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    cache = dsa.LatentCache(t(8, 512), t(8, 64))
    seqs = dsa.Seqs([0, 2], [0, 8], [6])
    with pytest.raises(ValueError, match="no words"):
        dsa.dsa_tree_mla_fwd(t(2, 4, 128), t(2, 4, 64), cache, t(4, 128, 512), t(4, 512, 128), seqs, 0.1,
                             tree_mask=torch.zeros(2, 0, dtype=torch.int64))


def test_rows_moved_at_the_end_of_32_bits():
    """Sequences that share their pages may have more rows together than the cache."""
    S = 2 ** 30 - 1
    seqs = _seqs([S, S], [S, S], [0, 0])
    pages = _pages(page_size=1 << 20, n_pages=0, width=1 << 11, ld_table=1 << 11)
    for call in (_write, _read):
        assert call(seqs=seqs, pages=pages) == DSA_ERR_UNSUPPORTED
    assert dsa.last_launch_count() == 0


@pytest.mark.parametrize("q,k", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 30, 2 ** 30), (2 ** 31 - 1024, 0),
                                 (1, 2 ** 31 - 1025)])
@pytest.mark.parametrize("D,d_r", [(128, 64), (8, 0), (7, 0), (512, 64)])
def test_head_counts_at_the_end_of_32_bits(q, k, D, d_r):
    """The heads of q and k together are counted in 32 bits: past them the call is refused, whatever the kernel.  (Heads
    of eight bf16 values would fit the GPU.)"""
    over = dict(ld_x=D * (1 << 31), ld_y=D * (1 << 31), hd_x=D, hd_y=D)
    assert _norm(q=_heads(n_heads=q, **over), k=_heads(n_heads=k, **over), D=D, d_r=d_r) == DSA_ERR_UNSUPPORTED
    assert dsa.last_launch_count() == 0


def test_rows_normed_at_the_end_of_32_bits():
    S = 2 ** 30 - 1
    assert _norm(q=_heads(n_heads=1), seqs=_seqs([S, S], [S, S], [0, 0]), n_pos=2 ** 30) == DSA_ERR_UNSUPPORTED
    assert dsa.last_launch_count() == 0


@pytest.mark.parametrize("part", ["tree_mla", "tree_mla_tc", "latent_cache", "head_norm"])
def test_no_host_memory_is_allocated(part):
    """The library's contract: what these parts import from C++ and C holds no allocation."""
    obj = os.path.join(os.path.dirname(dsa.__file__), "_build", part + ".o")
    nm = shutil.which("nm")
    if nm is None or not os.path.exists(obj):
        pytest.skip("no objects to look at")
    names = subprocess.run([nm, "-u", obj], check=True, capture_output=True, text=True).stdout.split()
    assert any("cudaLaunchKernel" in n for n in names)  # these are the imports
    bad = [n for n in names if n.startswith(("_Znw", "_Zna")) or n in ("malloc", "calloc", "realloc", "cudaMalloc", "cudaHostAlloc")]
    assert not bad, bad


def test_batches_of_any_sequence_of_numbers():
    """Lists, tuples, ranges, arrays, tensors and bytes of numbers describe the same batch."""
    want = [0, 3, 4], [0, 9, 16], [6, 6]
    for make in (list, tuple, lambda v: array.array("q", v), np.array, lambda v: np.array(v, dtype=np.float32), torch.tensor,
                 bytes, bytearray, lambda v: [torch.tensor(x) for x in v], lambda v: [float(x) for x in v]):
        s = dsa.Seqs(*(make(v) for v in want))
        assert [list(a[:n]) for a, n in ((s.struct.cu_q, 3), (s.struct.cu_k, 3), (s.struct.start_pos, 2))] == list(want)
        assert (s.B, s.total_q, s.total_k, s.max_S) == (2, 4, 16, 9)
    assert list(dsa.Seqs(range(5), range(0, 50, 10), [9] * 4).struct.cu_k[:5]) == [0, 10, 20, 30, 40]
    assert dsa.Seqs(b"\0\0\0\0\0", b"\0\1\2\3\4", b"\0\0\0\0").total_k == 4  # four bytes are four numbers


def test_the_longest_sequence_is_looked_for_once():
    s = dsa.Seqs([0, 1, 2], [0, 9, 16], [8, 6])
    assert s.max_S == 9 and "max_S" in vars(s)
    assert dsa.Seqs([0], [0], []).max_S == 0
