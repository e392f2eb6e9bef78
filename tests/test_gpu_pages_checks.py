"""Which entries the page bookkeeping looks at: those that a call shares, lets go or takes, no others."""
import pytest

from tests.test_gpu_pages import _i32, _refused, _state, pa  # noqa: F401

pytestmark = pytest.mark.gpu


def test_entries_that_stay_are_not_looked_at(pa):
    st = _state(4, 8, [40, 33], 16, 10, 9)
    first = st.p.tables[0][0]
    for bad in (-1, len(st.p.refs), 2 ** 31 - 1):
        st.tables[0, 0] = st.p.tables[0][0] = bad
        n = st.p.lens[0] + 16
        pa.pa_grow_sequences(st.tables, st.lens, _i32([0]), _i32([n]), *st.args())
        st.p.grow([0], [n])
        st.same()
        pa.pa_trim_sequences(st.tables, st.lens, _i32([0]), _i32([n - 15]), *st.args())
        st.p.end([0], [n - 15])
        st.same()
        # sharing it or letting it go
        _refused(pa, st, lambda: pa.pa_fork_sequences(st.tables, st.lens, _i32([0]), _i32([2]),
                                                      *st.args()))
        _refused(pa, st, lambda: pa.pa_free_sequences(st.tables, st.lens, _i32([1, 0]), *st.args()))
        _refused(pa, st, lambda: pa.pa_trim_sequences(st.tables, st.lens, _i32([0]), _i32([0]),
                                                      *st.args()))
    st.tables[0, 0] = st.p.tables[0][0] = first
    # a free block that is not taken
    st.free[0] = -7
    pa.pa_grow_sequences(st.tables, st.lens, _i32([1]), _i32([50]), *st.args())
    st.p.free[0] = -7
    st.p.grow([1], [50])
    st.same()
    n = st.count.item() * 16
    _refused(pa, st, lambda: pa.pa_grow_sequences(st.tables, st.lens, _i32([3]), _i32([n]), *st.args()))
    assert pa.pa_device_status() == pa.PA_OK
