"""CPU-only: the binding's and the library's edges around the tree and sparse operators."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

from test_masked_cpu import UNSUPPORTED, _accept, _err, _move, _select

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_187_gb300 import build
    build.build()
    import paged_kv_cache_187_gb300 as pkg
    return pkg


def test_the_allocator_and_the_raw_library_need_no_torch(pa):
    code = """
        import sys
        sys.modules["torch"] = None          # importing it raises
        import numpy as np
        import paged_kv_cache_187_gb300 as pa
        assert pa.raw().pa_version() > 0
        alloc = pa.PagedAllocator(10, 16, 3)
        alloc.pa_alloc_add_seq(1, 40)
        alloc.pa_alloc_append(1)
        assert alloc.num_free == 7
        assert pa.pa_decode_tree_workspace_size(100, 3, 8, 2, 128, 900) > 0
        assert pa.pa_select_blocks_workspace_size(3, 1, 2, 16, 900) > 0
        try:
            pa.pa_key_bounds(*[np.zeros((1, 2, 3, 4))] * 5, 1)
        except ImportError:
            pass
        else:
            raise AssertionError("a call with tensors")
    """
    subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT, check=True)


def test_torch_is_looked_up_at_the_first_call_with_tensors(pa):
    code = """
        import paged_kv_cache_187_gb300._binding as B, sys
        assert "torch" not in sys.modules and type(B.torch) is B._Torch
        assert B.torch.float16.itemsize == 2
        import torch
        assert B.torch is torch and B._address_of is torch.Tensor.data_ptr
        t = torch.zeros((2, 3))
        c = B._Call.__new__(B._Call)
        c.dev = -1                            # (the device of the host's tensors)
        assert list(c.pools((t, t), t.shape, t.dtype)) == [t.data_ptr()] * 2
    """
    subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT, check=True)


def test_pools_before_torch_is_looked_up(pa):
    code = """
        import torch
        import paged_kv_cache_187_gb300._binding as B
        assert type(B.torch) is B._Torch
        t = torch.zeros((2, 3))
        c = B._Call.__new__(B._Call)
        c.dev = -1
        assert list(c.pools((t, t), t.shape, t.dtype)) == [t.data_ptr()] * 2
    """
    subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT, check=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("wrong", [dict(out=(5, 4, 32)), dict(lens=(1, 1)), dict(starts=(3,)), dict(mask=(4, 1))])
def test_shape_errors_name_the_tree(pa, monkeypatch, fp8, wrong):
    import paged_kv_cache_187_gb300._binding as B

    class Here(B._Call):       # a machine without a GPU has no current device
        def __init__(self):
            self.dev = 0

    monkeypatch.setattr(B, "_Call", Here)
    shapes = dict(out=(5, 4, 64), q=(5, 4, 64), k=(9, 2, 16, 64), v=(9, 2, 16, 64), tables=(1, 4), lens=(1,),
                  starts=(2,), mask=(5, 1))
    args = [torch.zeros(x) for x in {**shapes, **wrong}.values()]
    with pytest.raises(ValueError, match="^decode_tree: "):
        (pa.pa_decode_tree_fp8 if fp8 else pa.pa_decode_tree)(*args, 64, 0.1, *([0.5, 0.5] if fp8 else []))
    if "mask" not in wrong:
        with pytest.raises(ValueError, match="^prefill: "):
            (pa.pa_prefill_fp8 if fp8 else pa.pa_prefill)(*args[:-1], 64, 0.1, *([0.5, 0.5] if fp8 else []))


@pytest.mark.parametrize("kw", [dict(), dict(first=2 ** 31 - 12), dict(first=0, last=2 ** 30)])
@pytest.mark.parametrize("n", [2 ** 30 + 1, 2 ** 31 - 1])
def test_lists_of_blocks_past_32_bit_steps_are_refused(pa, n, kw):
    kw = {k: min(x, n) for k, x in {**dict(first=1, last=0), **kw}.items()}
    assert _select(pa.raw(), n=n, **kw) == UNSUPPORTED
    assert "num_selected" in _err(pa.raw())


@pytest.mark.parametrize("most", [2 ** 30 + 1, 2 ** 31 - 1])
def test_paths_past_32_bit_steps_are_refused_by_the_accept(pa, most):
    assert _accept(pa.raw(), most=most) == UNSUPPORTED
    assert "max_accepted" in _err(pa.raw())


@pytest.mark.parametrize("kw,word", [(dict(most=2 ** 30 + 1), "max_accepted"), (dict(most=2 ** 31 - 1), "max_accepted"),
                                     (dict(Hkv=2 ** 31 - 1, D=8), "heads"), (dict(Hkv=2 ** 30 + 1, D=8), "heads")])
def test_paths_and_rows_past_32_bit_steps_are_refused_by_the_move(pa, kw, word):
    assert _move(pa.raw(), **kw) == UNSUPPORTED
    assert word in _err(pa.raw())
