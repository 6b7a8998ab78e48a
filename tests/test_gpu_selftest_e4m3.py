"""Tensor-core operand layouts of e4m3 tiles, checked on the GPU against host math (small integers, exact).

Images are built on the host from the layout definitions: rows of 128 bytes in the 128-byte swizzle (16-byte chunk c of
row r sits at chunk c ^ (r % 8)), and unswizzled core matrices of 8 keys x 16 bytes.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_248_gb300 as m
    m.lib()
    return m


def small_ints(shape, seed):
    return np.random.default_rng(seed).integers(-3, 4, size=shape).astype(np.float32)


def codes(a):
    return torch.from_numpy(a).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def swizzled(x):
    """[R][128] bytes, chunk c of row r at c ^ (r % 8)."""
    img = np.zeros((x.shape[0], 8, 16), np.uint8)
    for r in range(x.shape[0]):
        for c in range(8):
            img[r, c ^ (r % 8)] = x[r, 16 * c:16 * c + 16]
    return img.reshape(-1)


def columns16(p):
    """[K][N] bytes as [N / 16][K][16]: core matrices of 8 keys, 128 bytes apart along K, K * 16 along N."""
    k, n = p.shape
    return np.ascontiguousarray(p.reshape(k, n // 16, 16).transpose(1, 0, 2)).reshape(-1)


def run(pkv, n, a_mn, b_mn, a, b, a_img, b_img, a_step, b_step):
    off = [i * a_step for i in range(4)] + [0] * 4 + [i * b_step for i in range(4)] + [0] * 4
    params = [128, n, a_mn, b_mn, *a, *b, a_img.nbytes, b_img.nbytes, 4] + off
    d = torch.full((128, n), float("nan"), device="cuda")
    pkv.pkv_umma8_selftest(params, torch.from_numpy(a_img).cuda(), torch.from_numpy(b_img).cuda(), d)
    torch.cuda.synchronize()
    assert pkv.pkv_get_last_error() == 0
    return d.cpu().numpy()


@pytest.mark.parametrize("n", [16, 32, 64])
def test_keys_by_queries(pkv, n):
    # S^T = K Q^T: A = K tile [128 keys][128 d], B = Q [n rows][128 d], both K-major
    k, q = small_ints((128, 128), 1), small_ints((n, 128), 2)
    d = run(pkv, n, 0, 0, (2, 16, 1024), (2, 16, 1024), swizzled(codes(k)), swizzled(codes(q)), 32, 32)
    np.testing.assert_array_equal(d, k @ q.T)


@pytest.mark.parametrize("n", [16, 32, 48, 96])
def test_values_by_weights(pkv, n):
    # O^T = V^T P^T: A = V tile [128 keys][128 d] read MN-major, B = P [128 keys][n] MN-major without a swizzle
    v, p = small_ints((128, 128), 3), small_ints((128, n), 4)
    d = run(pkv, n, 1, 1, (2, 16384, 1024), (0, 128, 2048), swizzled(codes(v)), columns16(codes(p)), 4096, 512)
    np.testing.assert_array_equal(d, v.T @ p)
