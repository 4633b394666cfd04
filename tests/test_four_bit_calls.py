"""Calls of the 4-bit operators and the code scoring that their documentation
allows or refuses, found on the host before any device call (no GPU needed)."""
import pytest

ARG = -1
A = [0x1000000 * (i + 1) for i in range(16)]  # far apart, 16-byte aligned stand-ins, never dereferenced


@pytest.fixture(scope="module")
def lib():
    import ar_decode_step_gb300.build as b
    b.build()
    import ar_decode_step_gb300 as m
    return m.load()


SCORE = dict(z=A[0], ld=8208, codes=A[1], rows=4, n_cb=8, V=1026, T=1.0, top=5, lp=A[2], ent=A[3], at=A[4],
             at_lp=A[5], stream=None)


def test_code_logprobs_of_no_rows_wants_no_memory(lib):
    """An empty tensor's address is NULL: with no rows nothing is read or written.
    The sizes are checked all the same."""
    none = dict(SCORE, z=None, codes=None, rows=0, lp=None, ent=None, at=None, at_lp=None)
    assert lib.tts_code_logprobs(*none.values()) == 0
    assert lib.tts_code_logprobs(*dict(none, top=0).values()) == 0
    for bad in (dict(V=1), dict(n_cb=9), dict(top=33), dict(T=0.0), dict(ld=8207)):
        assert lib.tts_code_logprobs(*dict(none, **bad).values()) == ARG, bad
