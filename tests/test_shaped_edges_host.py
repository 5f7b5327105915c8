"""Edges of the shaped entry points without a GPU."""
import glob
import os
import re

import pytest
import torch

from exact_io_aware_tmem_b200 import _abi, attention


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_tmem_b200 import build
    build.build()
    return _abi.lib()


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), _abi.FA_OK), (dict(o=None), _abi.FA_ERR_INVALID_ARG),
    (dict(weights=None), _abi.FA_ERR_INVALID_ARG), (dict(slots=99), _abi.FA_ERR_INVALID_ARG),
    (dict(ws=None), _abi.FA_ERR_INVALID_ARG), (dict(ws=264), _abi.FA_ERR_INVALID_ARG),
    (dict(ws_bytes=1), _abi.FA_ERR_INVALID_ARG), (dict(H=130), _abi.FA_ERR_UNSUPPORTED),
    (dict(D=96), _abi.FA_ERR_UNSUPPORTED), (dict(max_len=0), _abi.FA_ERR_INVALID_ARG)])
def test_selftest_decode_finish_arguments(lib, kw, code):
    a = dict(o=256, lse=256, lens=256, B=2, q_len=1, H=4, H_kv=2, D=64, max_len=100, weights=256,
             slots=100, ws=256, ws_bytes=1 << 30)
    a.update(kw)
    assert lib.fa_selftest_decode_finish(*a.values(), None) == code


def test_kernels_that_start_early_take_no_restrict_pointers():
    # Such a kernel starts before the one ahead of it in the stream has ended: a pointer
    # that promises memory nobody writes meanwhile would allow non-coherent loads of it.
    csrc = os.path.join(os.path.dirname(_abi.__file__), "csrc")
    early = []
    for path in glob.glob(os.path.join(csrc, "*.cu")):
        for kernel in open(path).read().split("__global__")[1:]:
            body = kernel[:kernel.index("\n}\n")]
            if "wait_for_primary();" in body:
                early.append(re.search(r"(\w+_kernel)\(", body).group(1))
                assert "__restrict__" not in body[:body.index(") {")], early[-1]
    assert sorted(early) == ["finish_kernel", "move_kernel", "shaped_bwd_kernel"]


def test_stream_without_the_private_name(monkeypatch):
    class Stream:
        cuda_stream = 4711
    asked = []
    monkeypatch.setattr(attention, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: asked.append(d) or Stream)
    assert attention._stream(torch.device("cuda", 3)) == 4711 and asked == [3]
