"""A warp of the paged attention whose wait for a copy runs out: it waits for nothing more but the copies that it has in
flight, every stage at the parity that the stage is in, the call is flagged as timed out, all other units have their
results and the counters in the workspace are zero again, so that the next call is right. The wait is made to report that it ran out (tests/ring_give_up.cu); the copy
itself lands, and no wait is longer than the others."""
import ctypes
import os
import subprocess

import pytest
import torch

import compressed_decode_attention_equal_b200 as skv
from compressed_decode_attention_equal_b200 import _lib
from compressed_decode_attention_equal_b200.build import CSRC, INCLUDE
from test_gpu_cache import BF, F32, i32, make, rand

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
KINDS = {0: (BF, "e4m3", 128), 1: (BF, "raw", 64), 2: (F32, "raw", 64)}


@pytest.fixture(scope="module")
def helper(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("ring") / "libring_give_up.so")
    subprocess.run([os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc"), "-gencode", "arch=compute_100a,code=sm_100a", "-O3",
                    "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC, "-o", so,
                    os.path.join(HERE, "ring_give_up.cu")], check=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("B,Hkv,G,length,at", [(2, 2, 7, 60000, (0, 1, 2, 3, 4)), (512, 24, 1, 300, (0, 1, 7, 30, 61))])
def test_a_warp_that_gives_up_leaves_everything_in_order(helper, kind, B, Hkv, G, length, at):
    dtype, fmt, d = KINDS[kind]
    lens = [length - b % 100 for b in range(B)]
    g = torch.Generator().manual_seed(kind)
    cache, table = make(1, Hkv, d, dtype, fmt, [length])
    skv.cache_append(rand(g, length, Hkv, d, dtype=dtype).cuda(), rand(g, length, Hkv, d, dtype=dtype).cuda(), cache, table, i32([0]))
    table = table.expand(B, -1).contiguous()
    q = torch.randn(B, 1, G * Hkv, d, generator=g).to(dtype).cuda()
    n = i32(lens)
    want, want_lse = skv.paged_attn(q, cache, table, n)
    flags, counters = torch.zeros(64, dtype=torch.int32, device="cuda"), torch.zeros((1 << 16) + 1024, dtype=torch.int32, device="cuda")
    part_o, part_l = torch.empty(1024 * 8 * d, device="cuda"), torch.empty(1024 * 8, device="cuda")
    result = (ctypes.c_int * 4)()
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731

    def run(block, warp, at):
        out, lse = torch.full_like(q, 7.0), torch.full((B, 1, G * Hkv), 7.0, device="cuda")
        torch.cuda.synchronize()
        assert helper.run_give_up(kind, p(q), p(cache.pages), ctypes.c_int64(cache.num_pages), p(table), table.shape[1], p(n), p(out),
                                  p(lse), p(flags), p(counters), p(part_o), p(part_l), B, G * Hkv, Hkv, block, warp, at, result) == 0
        got = int(flags[0])
        flags.zero_()
        assert not counters.any()
        return out, lse, got

    stages = 2
    for block, warp, i in [(0, 0, at[0]), (3, 1, at[1]), (77, 0, at[2]), (77, 1, at[3]), (147, 0, at[4])]:
        out, lse, got = run(block, warp, i)
        waits, gave_up, drained, wrong = result
        assert gave_up == 1 and waits == i + 1 and got == _lib.FLAG_TIMEOUT, (list(result), got)
        assert 1 <= drained <= stages and wrong == 0, list(result)
        # units in order: those that differ are neighbours, the pieces of one CTA
        differ = (out != want).view(B * Hkv, -1).any(1) | (lse != want_lse).view(B * Hkv, -1).any(1)
        where = differ.nonzero().flatten()
        assert len(where) and int(where[-1] - where[0]) <= 100
        out, lse, got = run(block, warp, -1)
        assert got == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
        assert result[1] == 0 and result[2] == 0 and result[3] == 0 and result[0] > i
