"""Products whose results hold more than 2^32 values or have long edges: the bound is that of
the launch, counted in the tiles that the call takes."""

import ctypes

import pytest
import torch

from _helpers import dev
from quantize_grouped_gemm_amd import b128, moe

BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def test_what_one_launch_holds_is_accepted():
    """The check of the grid comes before that of `out`, which is missing here, so that nothing can run."""
    L = moe.lib()
    p, none = ctypes.c_void_p(16), None
    err = lambda: L.mx_last_error().decode()

    def status(rc):
        if rc == 1:
            assert "out is NULL" in err()
        else:
            assert rc == 2 and "tiles" in err(), (rc, err())
        return rc

    mm = lambda M, N, K=128: status(L.mx_b128_mm(p, p, p, p, 1, M, N, K, 0, none, N, none))
    assert [mm(32768, 151936), mm(65536, 129280), mm(131072, 131072), mm(1 << 18, 1 << 18), mm(1, 1 << 29), mm(1 << 28, 8)] == [1] * 6
    assert [mm(1 << 19, 1 << 20), mm(1 << 28, 1 << 18), mm(1 << 20, 1 << 18)] == [2] * 3
    grouped = lambda E, cap, N, K=128: status(L.mx_b128_grouped_mm(p, p, p, p, p, E, cap, N, K, none, none, none))
    assert [grouped(32, 1 << 20, 7168), grouped(256, 1 << 21, 14336), grouped(1024, 1 << 22, 16384), grouped(1, 127, 1 << 26),
            grouped(1024, 1 << 16, 65536)] == [1] * 5
    assert [grouped(1, 127, 1 << 30), grouped(32, 1 << 26, 1 << 17), grouped(1024, 1 << 16, 1 << 18)] == [2] * 3
    wgrad = lambda E, N, K: status(L.mx_b128_grouped_mm_wgrad(p, p, p, p, p, E, 1024, N, K, 0, none, none, none))
    assert [wgrad(256, 14336, 7168), wgrad(1024, 7168, 4096), wgrad(1024, 1, 65552), wgrad(8, 1 << 20, 8192)] == [1] * 4
    assert [wgrad(1024, 65536, 4096), wgrad(1, 1 << 20, 1 << 20)] == [2] * 2


def _gen(seed):
    return torch.Generator(device=dev()).manual_seed(seed)


def _codes(shape, seed):
    """Finite E4M3 codes."""
    q = torch.randint(0, 254, shape, generator=_gen(seed), device=dev(), dtype=U8)
    return q.masked_fill_((q & 0x7F) == 0x7F, 0)


def _scales(shape, seed):
    return torch.rand(shape, generator=_gen(seed), device=dev())


@pytest.fixture
def room(gpu):
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_logits_of_a_large_vocabulary(room):
    M, N, K = 32768, 151936, 128
    qa, sa, qb, sb = _codes((M, K), 1), _scales((1, M), 2), _codes((N, K), 3), _scales((1, N // 128), 4)
    got = b128.scaled_mm(qa, sa, qb, sb)
    for lo in (0, M // 2, M - 512):
        ref = b128.scaled_mm(qa[lo:lo + 512], sa[:, lo:lo + 512].contiguous(), qb, sb)
        assert torch.equal(got[lo:lo + 512], ref)


@pytest.mark.gpu
def test_grouped_rows_of_a_long_batch(room):
    E, cap, N, K = 3, 1 << 20, 7168, 128
    qa, sa, qw, sw = _codes((cap, K), 1), _scales((1, cap), 2), _codes((E, N, K), 3), _scales((E, 1, N // 128), 4)
    ends = [300000, 300001, cap - 5000]
    got = b128.grouped_mm(qa, sa, qw, sw, torch.tensor(ends, dtype=I32, device=dev()))
    for e, (lo, hi) in enumerate(((299000, 300000), (300000, 300001), (cap - 6000, cap - 5000))):
        ref = b128.scaled_mm(qa[lo:hi], sa[:, lo:hi].contiguous(), qw[e], sw[e])
        # one block of 128: the same products whatever the tile, under scales multiplied in one order
        assert torch.equal(got[lo:hi], ref)
    assert torch.all(got[ends[-1]:] == 0)


@pytest.mark.gpu
def test_weight_gradient_of_long_edges(room):
    E, N, K = 1024, 1, 65552
    qg, sg, qx, sx = _codes((N, 256), 1), _scales((2, N), 2), _codes((K, 256), 3), _scales((2, K), 4)
    offs = torch.full((E,), 256, dtype=I32, device=dev())
    offs[:700] = 128
    offs[:3] = 0
    got = b128.grouped_mm_wgrad(qg, sg, qx, sx, offs)
    for e, b in ((3, 0), (700, 1)):
        cut = lambda q: q[:, 128 * b:128 * (b + 1)].contiguous()
        ref = b128.grouped_mm_wgrad(cut(qg), sg[b:b + 1].contiguous(), cut(qx), sx[b:b + 1].contiguous(),
                                    torch.tensor([128], dtype=I32, device=dev()))
        assert torch.equal(got[e], ref[0])
    got[3] = 0
    got[700] = 0
    assert torch.all(got == 0)
