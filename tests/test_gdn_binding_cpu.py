"""CPU checks of what the binding of the gated delta rule makes of its arguments."""
import numpy as np
import pytest
import torch

from recurrent_state_update_amd._ffi import lib
from recurrent_state_update_amd.pool import LayerWeights, Pool, _rows
from tests.test_gdn_cpu import OK, UNSUP, make, multi


@pytest.fixture
def layer():
    pool = Pool.allocate_gdn(1, 3, 3, 16, 32, 1, 4, device="cpu")
    cd = pool.conv_dim
    return pool, LayerWeights(-torch.ones(3), None, torch.zeros(3), torch.zeros(cd, 4), None)


def strides(pool, w, rows, u, a, b, o, exact=True):
    args = pool._gdn_rows(w, rows, *pool.split_qkv(u), a, b, o, exact)
    return args[1:10:2] + [args[12]]          # q, k, v, a, b and o


@pytest.mark.parametrize("rows", [0, 1])
def test_the_stride_of_a_single_row_is_its_width(layer, rows):
    """Whatever torch says it is: a view of a wider row, or of an expanded one."""
    pool, w = layer
    wide = torch.zeros(1, pool.conv_dim + 7)
    u, a, b, o = wide[:rows, :-7], wide[:rows, -7:-4], wide[:rows, -4:-1], wide[:rows, :48]
    assert strides(pool, w, rows, u, a, b, o) == [32, 32, 48, 3, 3, 48]
    assert strides(pool, w, rows, u.as_strided(u.shape, (0, 1)), a, b, o) == [32, 32, 48, 3, 3, 48]


def test_the_stride_of_several_rows_is_passed_on(layer):
    pool, w = layer
    wide = torch.zeros(2, pool.conv_dim + 7)
    n = wide.shape[1]
    assert strides(pool, w, 2, wide[:, :-7], wide[:, -7:-4], wide[:, -4:-1], wide[:, :48]) == [n] * 6


def test_an_empty_batch_takes_an_empty_checkpoint_table(layer):
    """No sequences: nothing to do, with a [0, max_ckpt] table as without one."""
    pool, w = layer
    none = np.zeros(0, np.int32)
    assert pool.gdn_workspace_size([0], ckpt_interval=16) == 0
    for table in (np.zeros((0, 3), np.int32), none, []):
        assert pool.gdn_workspace_size([0], ckpt_interval=16, ckpt_slots=table) == 0
        assert pool._ckpt_table(table, 0)[2] == 0
    assert pool._ckpt_table([[1, 2], [-1, 0]], 2)[2] == 2 and pool._ckpt_table([1, 2], 2)[2] == 1
    with pytest.raises(ValueError):
        pool._ckpt_table([[1, 2]], 0)
    with pytest.raises(ValueError):
        pool._ckpt_table([1, 2, 3], 2)


def test_the_workspace_query_names_a_type_it_does_not_take(layer):
    pool, _ = layer
    for dt in (torch.float16, torch.int32):
        with pytest.raises(TypeError, match="unsupported dtype"):
            pool.gdn_workspace_size([0, 5], io_dtype=dt)
        with pytest.raises(TypeError, match="unsupported dtype"):
            pool.gdn_workspace_size([0, 5], o_dtype=dt)


def test_strides_that_no_element_uses_are_not_looked_at():
    """A dimension of one element, or an empty tensor, may have any stride; others are refused."""
    assert _rows(torch.zeros(1, 6).t(), "a")[1] == 1                  # [6, 1]: one gate per row
    assert _rows(torch.zeros(8).as_strided((0, 4), (0, 0)), "q")[1] == 0
    assert _rows(torch.from_numpy(np.zeros((0, 5))), "q")
    for bad in (torch.zeros(4, 6).t(), torch.zeros(2, 3, 4), torch.zeros(4), torch.zeros(4, 6)[:, ::2]):
        with pytest.raises(ValueError):
            _rows(bad, "q")


def test_workspace_of_fp32_rows_against_bf16_rows():
    """What the header says of it, at the ends of the shapes."""
    ratio = []
    for hk, hv, dk in ((1, 64, 32), (16, 32, 128), (2, 8, 32), (8, 8, 256)):
        pool = Pool.allocate_gdn(1, 1, hv, 16, dk, hk, 4, device="cpu")
        size = lambda dt: pool.gdn_workspace_size([0, 64 * 400], io_dtype=dt, o_dtype=dt)
        ratio.append(size(torch.float32) / size(torch.bfloat16))
    assert 2.7 <= min(ratio) and max(ratio) <= 3.0, ratio


@pytest.mark.parametrize("heads,code", [(42, OK), (43, UNSUP)])
def test_drafts_up_to_the_last_byte_of_lds(heads, code):
    """Per token 2 dk + heads (dv + 2) + 1 floats: 3 x 13653 of them are 4 bytes below 160 KiB.  (No rows: nothing runs.)"""
    h = make(H=heads, P=320, N=64, G=1)
    width = heads * 320
    assert multi(h, batch=0, tokens=3, vs=width, qs=64, ks=64, os=width, as_=heads, bs=heads) == code
    lib().mamba2_pool_destroy(h)
