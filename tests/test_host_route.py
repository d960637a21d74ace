"""How the router spreads its tokens follows the number of multiprocessors, not a count made for one.  On the CPU."""
import pytest

from host_calls import run


@pytest.mark.parametrize("sms", [152, 100, 20])
def test_tokens_per_block_follow_the_multiprocessors(tmp_path, sms):
    run(tmp_path, f"""
sms = {sms}
fake.fake_multiprocessors(sms)
for T, blocks in ((128, 1), (129, 9), (16 * sms, sms), (16 * sms + 1, -(-(16 * sms + 1) // 64))):
    log()
    assert route(T, E=8) == 0
    launches = log('launch')
    assert [e[4] for e in launches] == [blocks] * (1 if T <= 128 else 2), (T, launches)
""")
