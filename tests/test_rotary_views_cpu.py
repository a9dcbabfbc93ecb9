"""Views of rotary positions that share memory, refused without a GPU."""
from tests.test_mixer_cpu import FAKE, MB, _rot, lib  # noqa: F401


def test_interleaved_heads_that_overlap():
    st = (4 * 2 * 96, 2 * 96, 96)          # a head of 64 in every 96
    one = dict(q=FAKE, q_out=FAKE, q_strides=st, q_out_strides=st, k_strides=st, k_out_strides=st, d=64)
    for off in (0, 32, 63, -32, 96 + 40, -96 - 40):      # k's heads over q's
        k = FAKE + 2 * off
        assert _rot(**one, k=k, k_out=k) == -2, off
    # other strides of tokens or batches: no common period
    for bad in ((4 * 2 * 96, 2 * 96 + 8, 96), (4 * 2 * 96 + 8, 2 * 96, 96)):
        assert _rot(**dict(one, k_strides=bad, k_out_strides=bad), k=FAKE + 2 * 64, k_out=FAKE + 2 * 64) == -2
    assert _rot(**dict(one, q_out=FAKE + 8 * MB), k=FAKE + 2 * MB, k_out=FAKE + 8 * MB + 64) == -2
