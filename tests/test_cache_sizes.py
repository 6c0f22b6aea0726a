"""Which kernel takes a call, asked of the C entry on the host: calls that the
tensor-core kernels can run do not fall to the general one.  No GPU needed."""

import ctypes

import pytest

import dequant_gemm_int4_b200 as q4
from dequant_gemm_int4_b200 import build as q4build
from test_cache_host import cache


@pytest.fixture(scope="module")
def L():
    q4build.build()
    return q4.lib()


@pytest.mark.parametrize("rows, q_heads, tokens, path", [
    (131072, 32, 262144, q4.PATH_AUTO), (131072, 32, 262144, q4.PATH_PREFILL),
    (262144, 64, 262144, q4.PATH_AUTO), (1 << 20, 32, 1 << 20, q4.PATH_PREFILL),
    (131072, 32, 1 << 20, q4.PATH_DECODE),
])
def test_large_prompts_take_a_tensor_core_kernel(L, rows, q_heads, tokens, path):
    size = ctypes.c_size_t(0)
    c = cache(pages=tokens // 64, page_size=64, heads=8, head_dim=128, group=128)
    rc = L.int4_cache_attention_workspace_size(c, 1, rows, q_heads, 1, tokens // 64, path, ctypes.byref(size))
    assert rc == q4.OK, L.int4_last_error()
    assert size.value > 0  # the general kernel needs none


def test_more_steps_than_32_bits_are_refused(L):
    size = ctypes.c_size_t(0)
    c = cache(pages=1 << 20, page_size=1024, heads=8, head_dim=128, group=128)
    for path in (q4.PATH_DECODE, q4.PATH_PREFILL):
        assert L.int4_cache_attention_workspace_size(c, 1, 1 << 24, 64, 1, 1 << 20, path,
                                                     ctypes.byref(size)) == q4.ERR_UNSUPPORTED


@pytest.mark.parametrize("head_dim, group, tiles", [(128, 32, False), (64, 32, False), (256, 32, False), (256, 256, False),
                                                    (128, 64, True), (128, 128, True), (64, 64, True), (96, 32, True)])
def test_row_tiles_of_32_where_they_do_not_spill(L, head_dim, group, tiles):
    """The workspace holds two pieces a block of the row tile's height: the same
    for 16 and 32 rows a head where both take tiles of 16."""
    sizes = []
    for rows in (16, 32):
        size = ctypes.c_size_t(0)
        c = cache(pages=64, page_size=64, heads=8, head_dim=head_dim, group=group)
        assert L.int4_cache_attention_workspace_size(c, 1, 32 * rows, 8, 32, 64, q4.PATH_DECODE,
                                                     ctypes.byref(size)) == q4.OK
        sizes.append(size.value)
    assert (sizes[0] != sizes[1]) == tiles


@pytest.mark.parametrize("head_dim, group, dtype, most", [
    (128, 128, 1, 96), (128, 128, 2, 96), (128, 64, 1, 96), (128, 64, 2, 128), (128, 32, 1, 64), (128, 32, 2, 80),
    (96, 96, 1, 96), (96, 32, 1, 96), (96, 32, 2, 96), (64, 64, 1, 112), (64, 32, 1, 112), (64, 32, 2, 112),
    (256, 256, 1, 1 << 20)])
def test_the_few_rows_kernel_is_taken_as_far_as_it_is_faster(L, head_dim, group, dtype, most):
    def ask(rows, path):
        size = ctypes.c_size_t(0)
        c = cache(pages=64, page_size=64, heads=8, head_dim=head_dim, group=group)
        rc = L.int4_cache_attention_workspace_size(c, dtype, 32 * rows, 8, 32, 64, path, ctypes.byref(size))
        return size.value if rc == q4.OK else None

    for rows in (1, 32, 64, 80, 96, 112, 128, 144, 256, 1000):
        few, many = ask(rows, q4.PATH_DECODE), ask(rows, q4.PATH_PREFILL)
        assert few != many
        assert ask(rows, q4.PATH_AUTO) == (few if rows <= most else many), rows
