"""Calls of the token preparation and of the attention behind a prefix that their documentation allows and that are easily
got wrong: raw stream handles, tensors that lie beside each other in one projection or cache, checked calls, and every
combination of launches with guard bytes around what it writes."""

import pytest

from test_qk_rope import Inputs

import scaled_dot_product_vt_gb300 as vt


@pytest.fixture(scope="module", autouse=True)
def _built():
    vt.build()
    vt.load()


# ---------------------------------------------------------------- raw stream handles

@pytest.mark.gpu
def test_the_raw_handle_of_the_default_stream():
    """stream=0 (torch.cuda.default_stream().cuda_stream) is the default stream, whichever one is current."""
    x = Inputs("bf16", 1, 2, 1, 20, 64, 64, seed=21)
    torch = x.torch
    seen = lambda: torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    for current in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(current):
            assert vt._elsewhere(seen, x.q, torch.cuda.default_stream().cuda_stream, (), {}) == 0
            assert vt._elsewhere(seen, x.q, side.cuda_stream, (), {}) == side.cuda_stream
            assert vt._elsewhere(seen, x.q, side, (), {}) == side.cuda_stream
    torch.cuda.synchronize()
    # the call reads what the stream wrote before it
    old = vt.qk_rope(x.q, x.k, x.freqs, x.pos, **x.form())
    torch.cuda._sleep(1 << 23)  # a few milliseconds
    x.pos.zero_()
    got = vt.qk_rope(x.q, x.k, x.freqs, x.pos, stream=0, **x.form())
    torch.cuda.synchronize()
    want = vt.qk_rope(x.q, x.k, x.freqs, x.pos, **x.form())
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not torch.equal(got[0], old[0])
