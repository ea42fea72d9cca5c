"""Sizes at the ends of what attention, rotary positions and AdamW serve; no call here gets as far as a launch."""
from test_attention_host import T, _rotary  # noqa: F401  (T: the fixture)


def test_rotary_heads_whose_count_does_not_fit_with_another(T):  # noqa: F811
    # heads of one element, all of which stay: runs of heads would be counted beyond 2^31
    some = (1 << 30) + 1
    for heads in (some, (1 << 31) - 1):
        assert _rotary(T, shape=(1, 1, heads, 1), axes=1, sections=(0,), xs=(heads, heads, 1), ys=(heads, heads, 1)) == 3
        assert T.convtranspose_last_error()
    assert _rotary(T, shape=(0, 1, 1 << 30, 1), axes=1, sections=(0,), xs=(1, 1, 1), ys=(1, 1, 1)) == 0
