"""Groups out of order in calls of several launches: whichever launch they concern, they are reported, and every
sequence is right. Tolerances are those of test_kv8_shared_gpu.py."""
import pytest

from test_kv8_shared_gpu import FEW, FORMS, MANY, Batch, _attend, _check, _q, _status

pytestmark = pytest.mark.gpu


@FORMS
@pytest.mark.parametrize("fill", [0, 0x3F, 0xFF])
def test_groups_of_another_launch_out_of_order(form, fill):
    """600 sequences are two launches; the second one's group is in order by itself, the two before it overlap. 8960 shared
    tokens and 40 of each sequence: what a block takes by itself where they are shared and what is spread where they are not."""
    import dense_bf16_gemm_02_gb300 as hk
    batch = Batch([(8960, [40] * 600)], 1, 64, 64)
    q = _q(batch.B, 1, 2, 64)
    got = _attend(batch, q, form=form, fill=fill, offsets=[0, 300, 200, 600], shared=[8960] * 3)
    assert _status() == hk.HK_ERR_INVALID_ARG
    _check(batch, q, got, form=form)
    got = _attend(batch, q, form=form, fill=fill)
    assert _status() == hk.HK_OK
    _check(batch, q, got, form=form)


@pytest.mark.parametrize("at", [5, 700, 1025, 1060, 1099])
def test_one_of_many_groups_out_of_order(at):
    """1100 groups, of which a launch plans for 512: one that no launch's sequences lead to is reported too."""
    import dense_bf16_gemm_02_gb300 as hk
    batch = Batch([(130, [1 + i % 3 for i in range(1200)])], 1, 64, 128)
    q = _q(batch.B, 1, 2, 64)
    groups = list(range(1024)) + [1024] * 66 + list(range(1024, 1034)) + [1200]        # (none of the middle ones is in order)
    if at < 1024:
        groups = list(range(1100)) + [1200]
        groups[at] = groups[at + 1] + 3
    elif at == 1099:
        groups = list(range(1100)) + [1199]
    else:
        groups[1025:1090] = [at - 1024] * 65
    got = _attend(batch, q, form=FEW, offsets=groups, shared=[128] * 1100)
    assert _status() == hk.HK_ERR_INVALID_ARG
    _check(batch, q, got, form=FEW)
    got = _attend(batch, q, form=FEW, offsets=list(range(1100)) + [1200], shared=[0] * 1100)
    assert _status() == hk.HK_OK
    _check(batch, q, got, form=FEW)


def test_many_rows_take_64_groups_of_two_launches():
    """Every group of the call is looked at by each of its launches: the largest number of them."""
    import dense_bf16_gemm_02_gb300 as hk
    batch = Batch([(300 + 40 * i, [1 + i % 5] * 10) for i in range(64)], 1, 64, 64)
    q = _q(batch.B, 1, 2, 64)
    _check(batch, q, _attend(batch, q, form=MANY), form=MANY)
    assert _status() == hk.HK_OK
    for at in (1, 30, 63):
        offsets = list(batch.offsets)
        offsets[at] = offsets[at + 1]
        got = _attend(batch, q, form=MANY, offsets=offsets)
        assert _status() == hk.HK_ERR_INVALID_ARG
        _check(batch, q, got, form=MANY)
